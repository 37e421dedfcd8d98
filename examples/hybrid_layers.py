"""A two-layer recurrent model served with this package's calls: one KDA layer and one state-space
layer, a prompt of packed sequences followed by single tokens.

    residual norm -> projection -> short convolution -> kda.fwd or kda.ssm -> gated norm -> projection

Every state (the convolution's last rows, the mixer's matrix) is handed from the prompt to the steps
and updated in place. Random weights; run it to see that steps after a prompt give what one longer
prompt gives:

    python examples/hybrid_layers.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_linear_attention_kda_gb300 as kda  # noqa: E402

BF16 = torch.bfloat16


class Layer:
    """What both layers share: the norm before the block and the convolution's taps."""

    def __init__(self, dim, conv_channels, gen):
        self.dim, self.gen = dim, gen
        self.norm = torch.ones(dim, device="cuda")
        self.taps = self.param(conv_channels, 4, scale=0.5)

    def param(self, *shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=self.gen, device="cuda") * scale).to(dtype)

    def proj(self, rows, cols):
        return self.param(cols, rows, scale=rows ** -0.5, dtype=BF16)


class KdaLayer(Layer):
    """q, k, v through the convolution, kda.fwd with its gate, a norm per head and a sigmoid gate."""

    def __init__(self, dim, heads, gen):
        self.H, self.inner = heads, heads * 128
        super().__init__(dim, 3 * self.inner, gen)
        self.w_in, self.w_out = self.proj(dim, 5 * self.inner + heads), self.proj(self.inner, dim)
        self.A_log, self.dt_bias = self.param(heads, scale=0.5), self.param(heads, 128, scale=0.1)
        self.head_norm = torch.ones(128, device="cuda")

    def states(self, n):
        return {"conv": torch.zeros(n, 3, 3 * self.inner, dtype=BF16, device="cuda"),
                "mixer": torch.zeros(n, self.H, 128, 128, device="cuda")}

    def __call__(self, h, st, cu):
        n = 3 * self.inner
        row = torch.nn.functional.pad(h @ self.w_in.T, (0, -self.H % 8))  # token rows keep 16-byte strides
        lead, step = row.shape[:-1], row.dim() == 2
        qkv = torch.empty(*lead, n, dtype=BF16, device=h.device)
        if step:
            kda.conv_step(row[..., :n], self.taps, qkv, st["conv"])
        else:
            kda.conv(row[..., :n], self.taps, qkv, initial_state=st["conv"], final_state=st["conv"], cu_seqlens=cu)
        heads = lambda t: t.unflatten(-1, (self.H, 128))  # noqa: E731
        q, k, v = (heads(t).contiguous() for t in qkv.split(self.inner, -1))
        g, beta = heads(row[..., n:n + self.inner]).contiguous(), row[..., 5 * self.inner:5 * self.inner + self.H].contiguous()
        out = torch.empty_like(q)
        gate = (self.A_log, self.dt_bias, -5.0)
        if step:
            kda.decode(q, k, v, g, beta, 128 ** -0.5, out, st["mixer"], *gate, qk_l2norm=True)
        else:
            kda.fwd(q, k, v, g, beta, 128 ** -0.5, out, *gate, initial_state=st["mixer"], final_state=st["mixer"], cu_seqlens=cu,
                    qk_l2norm=True)
        kda.gated_norm(out, heads(row[..., 4 * self.inner:5 * self.inner]), self.head_norm, out)
        return out.flatten(-2) @ self.w_out.T


class SsmLayer(Layer):
    """x | b | c through the convolution, kda.ssm, the gate ahead of a norm over the whole row."""

    def __init__(self, dim, heads, gen, P=64):
        self.H, self.P, self.inner = heads, P, heads * P
        super().__init__(dim, self.inner + 256, gen)
        self.w_in, self.w_out = self.proj(dim, 2 * self.inner + 256 + heads), self.proj(self.inner, dim)
        self.A_log = torch.log(1 + 15 * torch.rand(heads, generator=gen, device="cuda"))
        self.dt_bias, self.D = self.param(heads, scale=1.0) - 4, torch.ones(heads, device="cuda")
        self.row_norm = torch.ones(self.inner, device="cuda")

    def states(self, n):
        return {"conv": torch.zeros(n, 3, self.inner + 256, dtype=BF16, device="cuda"),
                "mixer": torch.zeros(n, self.H, self.P, 128, device="cuda")}

    def __call__(self, h, st, cu):
        n = self.inner + 256
        row = torch.nn.functional.pad(h @ self.w_in.T, (0, -self.H % 8))
        lead, step = row.shape[:-1], row.dim() == 2
        xbc = torch.empty(*lead, n, dtype=BF16, device=h.device)
        if step:
            kda.conv_step(row[..., :n], self.taps, xbc, st["conv"])
        else:
            kda.conv(row[..., :n], self.taps, xbc, initial_state=st["conv"], final_state=st["conv"], cu_seqlens=cu)
        x = xbc[..., :self.inner].unflatten(-1, (self.H, self.P))
        b, c = (xbc[..., self.inner + 128 * i:self.inner + 128 * (i + 1)].unflatten(-1, (1, 128)) for i in (0, 1))
        dt = row[..., n + self.inner:n + self.inner + self.H]
        out = torch.empty(*lead, self.H, self.P, dtype=BF16, device=h.device)
        if step:
            kda.ssm_step(x, dt, b, c, out, st["mixer"], self.A_log, self.D, self.dt_bias)
        else:
            tokens = x.shape[0] * x.shape[1]
            ws = torch.empty(kda.ssm_workspace_bytes(st["mixer"].shape[0], tokens, self.H, self.P), dtype=torch.uint8, device=h.device)
            kda.ssm(x, dt, b, c, out, self.A_log, self.D, self.dt_bias, initial_state=st["mixer"], final_state=st["mixer"],
                    cu_seqlens=cu, workspace=ws)
        rows = out.flatten(-2).unsqueeze(-2)
        kda.gated_norm(rows, row[..., n:n + self.inner].unsqueeze(-2), self.row_norm, rows, act="silu", gate_first=True)
        return rows.squeeze(-2) @ self.w_out.T


class Model:
    def __init__(self, dim=512, heads=4, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.layers = [KdaLayer(dim, heads, gen), SsmLayer(dim, 2 * heads, gen)]
        self.last_norm = torch.ones(dim, device="cuda")

    def states(self, n):
        return [layer.states(n) for layer in self.layers]

    def __call__(self, embedded, states, cu=None):
        """``embedded``: bf16 [1, T, dim] packed prompts with their ``cu``, or [S, dim] single tokens.
        Returns the normed last rows; ``states`` are updated in place."""
        residual = embedded.float()
        h = torch.empty_like(embedded)
        kda.residual_norm(torch.zeros_like(embedded), residual, None, self.layers[0].norm, h)
        for i, layer in enumerate(self.layers):
            y = layer(h, states[i], cu)
            norm = self.layers[i + 1].norm if i + 1 < len(self.layers) else self.last_norm
            kda.residual_norm(y, residual, residual, norm, h)
        return h


def packed(lengths):
    return torch.tensor([0] + list(lengths), dtype=torch.int64).cumsum(0).cuda()


def prompt_then_steps(model, rows, steps):
    """Prompts of all but the last ``steps`` tokens of every row, then single tokens: the steps' outputs."""
    states, cut = model.states(len(rows)), [r[:len(r) - steps] for r in rows]
    model(torch.cat(cut)[None], states, packed(len(r) for r in cut))
    return torch.stack([model(torch.stack([r[len(r) - steps + i] for r in rows]), states) for i in range(steps)], 1)


def whole_prompts(model, rows, steps):
    """The same tokens in one call: the outputs of every row's last ``steps`` tokens."""
    lengths = [len(r) for r in rows]
    out = model(torch.cat(rows)[None], model.states(len(rows)), packed(lengths))[0]
    return torch.stack([o[-steps:] for o in out.split(lengths)])


def main():
    model = Model()
    gen = torch.Generator(device="cuda").manual_seed(1)
    rows = [torch.randn(n, 512, generator=gen, device="cuda").to(BF16) for n in (37, 300, 5, 161)]
    a, b = prompt_then_steps(model, rows, 4), whole_prompts(model, rows, 4)
    kda.check_device_status()
    rel = float((a.float() - b.float()).norm() / b.float().norm())
    print(f"4 prompts, 4 steps each: steps against one longer prompt, relative difference {rel:.2e}")
    return rel


if __name__ == "__main__":
    main()
