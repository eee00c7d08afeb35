"""Two layers as they stand next to one another in a hybrid stack, in the three ways they are run: a
training step, the prefill of packed prompts into slot caches, and decode steps on those caches.

    x = x + recurrence(x):   u, r, i, z = projections of x
                             h = gated linear recurrence of u with gates from r and i
                             group norm of h, times silu(z), then the output projection
    x = x + attention(x):    q, k, v, z = projections of x
                             q, k normalised for each head and turned by their positions
                             o = linear attention of q, k, v; norm, gate and projection as above

    python -m chunked_gated_delta_gdn_gb300.examples.hybrid_block
"""
from __future__ import annotations

import torch
from torch import nn

import chunked_gated_delta_gdn_gb300 as gdn


class _Layer(nn.Module):
    """Input projection in parts, norm of groups times silu of a gate, output projection."""

    def __init__(self, dim, parts, width, groups, device, dtype):
        super().__init__()
        self.parts, self.groups = parts, groups
        self.inp = nn.Linear(dim, sum(parts), bias=False, device=device, dtype=dtype)
        self.out = nn.Linear(width, dim, bias=False, device=device, dtype=dtype)
        self.weight = nn.Parameter(torch.ones(width, device=device))

    def finish(self, o, z, train=False):
        norm = gdn.group_norm_act_trainable if train else gdn.group_norm_act
        shape = z.shape
        y = norm(o.reshape(-1, shape[-1]), self.groups, self.weight, gate=z.reshape(-1, shape[-1]).contiguous())
        return self.out(y.view(shape))


class RecurrentLayer(_Layer):
    """``dim`` -> ``dim`` over ``width`` channels; u, r and i are read where the projection left them."""

    def __init__(self, dim, width=128, groups=2, device="cuda", dtype=torch.bfloat16):
        super().__init__(dim, (width,) * 4, width, groups, device, dtype)
        # decays of open gates evenly from 0.9 to 0.999
        u = torch.linspace(0.9, 0.999, width, dtype=torch.float64)
        self.lam = nn.Parameter(torch.log(torch.expm1(-torch.log(u) / 8.0)).float().to(device))
        self.cache_shape = (width,)

    def forward(self, x, cu_seqlens=None, positions=None):
        u, r, i, z = self.inp(x).split(self.parts, -1)
        h, _ = gdn.gated_linear_recurrence_fused_gates_trainable(u, r, i, self.lam, cu_seqlens=cu_seqlens)
        return self.finish(h, z, train=True)

    @torch.no_grad()
    def prefill(self, x, cu_seqlens, positions, cache, slots):
        u, r, i, z = self.inp(x).split(self.parts, -1)
        h, _ = gdn.gated_linear_recurrence_fused_gates(u, r, i, self.lam, initial_state=cache,
                                                       output_final_state=True, cu_seqlens=cu_seqlens,
                                                       state_indices=slots)
        return self.finish(h, z)

    @torch.no_grad()
    def decode(self, x, positions, cache, slots):
        u, r, i, z = self.inp(x).split(self.parts, -1)
        return self.finish(gdn.gated_linear_recurrence_decode_fused_gates(u, r, i, self.lam, cache, slots), z)


class RotatedAttnLayer(_Layer):
    """Linear attention with Hv value heads of V and Hqk query / key heads of K, which are normalised with
    weights of their own and turned by their tokens' positions."""

    def __init__(self, dim, Hqk=2, Hv=4, K=64, V=64, device="cuda", dtype=torch.bfloat16):
        super().__init__(dim, (Hqk * K, Hqk * K, Hv * V, Hv * V), Hv * V, Hv, device, dtype)
        self.Hqk, self.Hv = Hqk, Hv
        self.q_weight = nn.Parameter(torch.ones(K, device=device))
        self.k_weight = nn.Parameter(torch.ones(K, device=device))
        freq = 10000.0 ** (-torch.arange(0, K, 2, dtype=torch.float64) / K)
        self.register_buffer("inv_freq", freq.float().to(device))
        h = torch.arange(Hv, dtype=torch.float64)
        self.register_buffer("log_decay", torch.log1p(-torch.exp2(-5.0 - h)).float().to(device))
        self.cache_shape = (Hv, K, V)

    def project(self, x):
        q, k, v, z = self.inp(x).split(self.parts, -1)
        heads = lambda t, H: t.unflatten(-1, (H, -1))
        return heads(q, self.Hqk), heads(k, self.Hqk), heads(v, self.Hv).contiguous(), z

    def forward(self, x, cu_seqlens=None, positions=None):
        q, k, v, z = self.project(x)
        q, k = gdn.qk_norm_rotate_trainable(q, k, self.inv_freq, positions, self.q_weight, self.k_weight)
        o, _ = gdn.chunk_linear_attn_trainable(q, k, v, self.log_decay, cu_seqlens=cu_seqlens)
        return self.finish(o, z, train=True)

    @torch.no_grad()
    def prefill(self, x, cu_seqlens, positions, cache, slots):
        q, k, v, z = self.project(x)
        q, k = gdn.qk_norm_rotate(q, k, self.inv_freq, positions, self.q_weight, self.k_weight)
        o, _ = gdn.chunk_linear_attn(q, k, v, self.log_decay, initial_state=cache, output_final_state=True,
                                     cu_seqlens=cu_seqlens, state_indices=slots)
        return self.finish(o, z)

    @torch.no_grad()
    def decode(self, x, positions, cache, slots):
        q, k, v, z = self.project(x)
        q, k = gdn.qk_norm_rotate(q, k, self.inv_freq, positions, self.q_weight, self.k_weight)
        return self.finish(gdn.linear_attn_decode(q, k, v, self.log_decay, cache, slots), z)


class HybridBlock(nn.Module):
    """A recurrent layer and an attention layer, each added to its input."""

    def __init__(self, dim, device="cuda", dtype=torch.bfloat16, **attn):
        super().__init__()
        self.layers = nn.ModuleList([RecurrentLayer(dim, device=device, dtype=dtype),
                                     RotatedAttnLayer(dim, device=device, dtype=dtype, **attn)])

    def caches(self, num_slots):
        return [torch.zeros(num_slots, *layer.cache_shape, device=self.layers[0].lam.device) for layer in self.layers]

    def forward(self, x, cu_seqlens=None, positions=None):
        """Training: x [B, T, dim], or [1, T, dim] with ``cu_seqlens`` and ``positions`` [1, T] int32;
        differentiable."""
        for layer in self.layers:
            x = x + layer(x, cu_seqlens, positions)
        return x

    def prefill(self, x, cu_seqlens, positions, caches, slots):
        """Packed prompts x [1, T, dim]; sequence i starts from slot ``slots[i]`` of every cache and leaves its
        states there."""
        for layer, cache in zip(self.layers, caches):
            x = x + layer.prefill(x, cu_seqlens, positions, cache, slots)
        return x

    def decode(self, x, positions, caches, slots):
        """The next token of each request: x [n, dim] at ``positions`` [n] int32, -1 slots are padding."""
        for layer, cache in zip(self.layers, caches):
            x = x + layer.decode(x, positions, cache, slots)
        return x


def packed(lens, device="cuda"):
    """cu_seqlens [N + 1] and positions [1, T] of packed sequences."""
    cu = torch.tensor([sum(lens[:n]) for n in range(len(lens) + 1)], dtype=torch.int32, device=device)
    pos = torch.cat([torch.arange(n, dtype=torch.int32, device=device) for n in lens])[None]
    return cu, pos


def main():
    torch.manual_seed(0)
    block = HybridBlock(256)
    opt = torch.optim.Adam(block.parameters(), lr=3e-3)
    x = torch.randn(2, 300, 256, device="cuda", dtype=torch.bfloat16)
    target = torch.randn_like(x)
    for step in range(3):
        loss = (block(x) - target).float().square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        print("step %d: loss %.4f" % (step, loss.item()))
    lens = [70, 1, 200]
    cu, pos = packed(lens)
    slots = torch.tensor([5, 0, 2], dtype=torch.int32, device="cuda")
    caches = block.caches(8)
    y = block.prefill(torch.randn(1, sum(lens), 256, device="cuda", dtype=torch.bfloat16), cu, pos, caches, slots)
    x = torch.stack([y[0, int(e) - 1] for e in cu[1:]])
    at = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for step in range(2):
        x = block.decode(x, at + step, caches, slots)
        print("token %d: norms %s" % (step, ["%.3f" % n for n in x.float().norm(dim=-1).tolist()]))


if __name__ == "__main__":
    main()
