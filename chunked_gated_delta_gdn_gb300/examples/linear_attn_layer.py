"""A layer of linear attention with a decay for each head, in the three ways it is run: a training
step, the prefill of packed prompts into a slot cache, and decode steps on that cache.

    q, k, v, z = projections of x
    o   = linear attention of q, k, v (heads of v share a head of q, k in groups)
    y   = group norm of o, a group a head, times silu(z), then the output projection

    python -m chunked_gated_delta_gdn_gb300.examples.linear_attn_layer
"""
from __future__ import annotations

import torch
from torch import nn

import chunked_gated_delta_gdn_gb300 as gdn


class LinearAttnLayer(nn.Module):
    """``dim`` -> ``dim`` with Hv value heads of V, Hqk query / key heads of K."""

    def __init__(self, dim, Hqk=2, Hv=4, K=64, V=64, device="cuda", dtype=torch.bfloat16):
        super().__init__()
        self.Hqk, self.Hv, self.K, self.V = Hqk, Hv, K, V
        self.splits = (Hqk * K, Hqk * K, Hv * V, Hv * V)
        self.inp = nn.Linear(dim, sum(self.splits), bias=False, device=device, dtype=dtype)
        self.out = nn.Linear(Hv * V, dim, bias=False, device=device, dtype=dtype)
        self.weight = nn.Parameter(torch.ones(Hv * V, device=device))
        self.bias = nn.Parameter(torch.zeros(Hv * V, device=device))
        # head h forgets a share 2^-(5 + h) of its state a token
        h = torch.arange(Hv, dtype=torch.float64)
        self.register_buffer("log_decay", torch.log1p(-torch.exp2(-5.0 - h)).float().to(device))

    def project(self, x):
        q, k, v, z = self.inp(x).split(self.splits, -1)
        heads = lambda t, H: t.unflatten(-1, (H, -1)).contiguous()
        return heads(q, self.Hqk), heads(k, self.Hqk), heads(v, self.Hv), z.contiguous()

    def forward(self, x, cu_seqlens=None):
        """Training: x [B, T, dim], or [1, T, dim] with ``cu_seqlens``; differentiable."""
        q, k, v, z = self.project(x)
        o, _ = gdn.chunk_linear_attn_trainable(q, k, v, self.log_decay, cu_seqlens=cu_seqlens)
        y = gdn.group_norm_act_trainable(o.flatten(0, 1).flatten(1), self.Hv, self.weight, self.bias,
                                         gate=z.flatten(0, 1))
        return self.out(y.view(*x.shape[:2], -1))

    def _finish(self, o, z):
        return self.out(gdn.group_norm_act(o.flatten(-2).view(z.shape), self.Hv, self.weight, self.bias, gate=z))

    @torch.no_grad()
    def prefill(self, x, cu_seqlens, cache, slots):
        """Packed prompts x [1, T, dim]; sequence i starts from slot ``slots[i]`` of ``cache``
        [num_slots, Hv, K, V] fp32 and leaves its state there."""
        q, k, v, z = self.project(x)
        o, _ = gdn.chunk_linear_attn(q, k, v, self.log_decay, initial_state=cache, output_final_state=True,
                                     cu_seqlens=cu_seqlens, state_indices=slots)
        return self._finish(o[0], z[0])[None]

    @torch.no_grad()
    def decode(self, x, cache, slots):
        """The next token of each request: x [n, dim], -1 slots are padding."""
        q, k, v, z = self.project(x)
        return self._finish(gdn.linear_attn_decode(q, k, v, self.log_decay, cache, slots), z)


def main():
    torch.manual_seed(0)
    layer = LinearAttnLayer(256)
    # a training step on two rows of 300 tokens
    opt = torch.optim.Adam(layer.parameters(), lr=3e-3)
    x = torch.randn(2, 300, 256, device="cuda", dtype=torch.bfloat16)
    target = torch.randn_like(x)
    for step in range(3):
        loss = (layer(x) - target).float().square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        print("step %d: loss %.4f" % (step, loss.item()))
    # three prompts into slots 5, 0 and 2, then two tokens each
    lens = [70, 1, 200]
    cu = torch.tensor([0, 70, 71, 271], dtype=torch.int32, device="cuda")
    slots = torch.tensor([5, 0, 2], dtype=torch.int32, device="cuda")
    cache = torch.zeros(8, layer.Hv, layer.K, layer.V, device="cuda")
    y = layer.prefill(torch.randn(1, sum(lens), 256, device="cuda", dtype=torch.bfloat16), cu, cache, slots)
    x = torch.stack([y[0, int(e) - 1] for e in cu[1:]])
    for step in range(2):
        x = layer.decode(x, cache, slots)
        print("token %d: norms %s" % (step, ["%.3f" % n for n in x.float().norm(dim=-1).tolist()]))


if __name__ == "__main__":
    main()
