"""A linear-attention block as a language model runs it, on the library's operators.

    r = residual + x;  u = norm(r)                                   ssm_add_norm_fwd
    q, k, v, z, a = split(W_in u);  g = -softplus(a + decay_bias)
    y = linear attention(q, k, v, g)                                 ssm_linattn_fwd / _state_update
    out = W_out (norm_per_head(y) * silu(z))                         ssm_gated_norm_fwd

* ``prompt`` runs a whole prompt (dense products) and leaves the state;
* ``token`` runs one token from it, with the projections in 4 bits (ssm_q4_matvec);
* ``gradients`` is the block's backward pass (ssm_*_bwd), recomputing what it needs.

Run:  python examples/linattn_block.py   (an MI355X; prints what it checked and timed)
"""
import os
import sys
import time

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sequence_scan_amd as ssm  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


def dense(codes, scales, zeros, group):
    """The bf16 matrix that a 4-bit one stands for."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(1).float().unflatten(1, (-1, group))
    return ((c - zeros[..., None].float()) * scales[..., None].float()).flatten(1).to(BF16)


class LinAttnBlock:
    """One block: ``width`` channels, ``heads`` heads of ``dim`` values, q and k shared by
    heads / groups heads each."""

    def __init__(self, width=1024, heads=8, groups=2, dim=64, group=64, seed=0, device="cuda"):
        r = torch.Generator(device="cpu").manual_seed(seed)
        self.H, self.G, self.d, self.group = heads, groups, dim, group
        self.sizes = [groups * dim, groups * dim, heads * dim, heads * dim, heads]
        rows = -(-sum(self.sizes) // 8) * 8          # q, k, v rows are multiples of 8 elements
        w_in = torch.randn(rows, width, generator=r).to(device) * width ** -0.5
        w_out = torch.randn(width, heads * dim, generator=r).to(device) * (heads * dim) ** -0.5
        self.in4 = ssm.ssm_q4_quantize(w_in, group, BF16)
        self.out4 = ssm.ssm_q4_quantize(w_out, group, BF16)
        self.w_in, self.w_out = dense(*self.in4, group), dense(*self.out4, group)
        self.norm_weight = (1 + 0.1 * torch.randn(width, generator=r)).to(device)
        self.head_weight = (1 + 0.1 * torch.randn(heads * dim, generator=r)).to(device)
        self.decay_bias = torch.linspace(-5, -1, heads).to(device)

    def _split(self, p):
        q, k, v, z, a = p[..., :sum(self.sizes)].split(self.sizes, -1)
        H, G, d = self.H, self.G, self.d
        return (q.unflatten(-1, (G, d)), k.unflatten(-1, (G, d)), v.unflatten(-1, (H, d)), z,
                -F.softplus(a.float() + self.decay_bias))

    def prompt(self, x, residual, state=None):
        """x, residual [batch, seqlen, width] -> out, the new residual, the last state."""
        B, L, D = x.shape
        u, r = ssm.ssm_add_norm_fwd(x, residual, self.norm_weight)
        q, k, v, z, g = self._split((u.view(B * L, D) @ self.w_in.t()).view(B, L, -1))
        last = torch.empty(B, self.H, self.d, self.d, device=x.device)
        y = ssm.ssm_linattn_fwd(q, k, v, g, initial_state=state, last_state=last)
        o = ssm.ssm_gated_norm_fwd(y.view(B, L, -1), z, self.head_weight, ngroups=self.H, gate_first=False)
        return (o.view(B * L, -1) @ self.w_out.t()).view(B, L, D), r, last

    def token(self, x, residual, state):
        """x, residual [batch, width]; ``state`` moves on in place and ``residual`` is replaced."""
        u, r = ssm.ssm_add_norm_fwd(x, residual, self.norm_weight, residual_out=residual)
        q, k, v, z, g = self._split(ssm.ssm_q4_matvec(u, *self.in4))
        y = ssm.ssm_linattn_state_update(state, q.contiguous(), k.contiguous(), v.contiguous(), g)
        o = ssm.ssm_gated_norm_fwd(y.flatten(1), z, self.head_weight, ngroups=self.H, gate_first=False)
        return ssm.ssm_q4_matvec(o, *self.out4), r

    def gradients(self, x, residual, dout, dresidual=None):
        """The gradients of x, residual and the parameters, given those of the block's two
        outputs (float32 residual stream)."""
        B, L, D = x.shape
        u, r = ssm.ssm_add_norm_fwd(x, residual, self.norm_weight)
        u2 = u.view(B * L, D)
        p = (u2 @ self.w_in.t()).view(B, L, -1)
        q, k, v, z, g = self._split(p)
        y = ssm.ssm_linattn_fwd(q, k, v, g).view(B, L, -1)
        o = ssm.ssm_gated_norm_fwd(y, z, self.head_weight, ngroups=self.H, gate_first=False)
        d2 = dout.view(B * L, D)
        do = (d2 @ self.w_out).view(B, L, -1)
        gn = ssm.ssm_gated_norm_bwd(do, y, z, self.head_weight, ngroups=self.H, gate_first=False)
        la = ssm.ssm_linattn_bwd(q, k, v, g, gn["dx"].view(B, L, self.H, self.d))
        a = p[..., sum(self.sizes[:4]):sum(self.sizes)].float() + self.decay_bias
        da = -la["dlog_decay"] * torch.sigmoid(a)
        pad = p.new_zeros(B, L, p.shape[-1] - sum(self.sizes))
        dp = torch.cat((la["dq"].flatten(2), la["dk"].flatten(2), la["dv"].flatten(2), gn["dz"], da.to(p.dtype), pad), -1)
        dp = dp.view(B * L, -1)
        an = ssm.ssm_add_norm_bwd((dp @ self.w_in).view(B, L, D), r, self.norm_weight, dresidual_out=dresidual, x=x)
        return {"x": an["dx"], "residual": an["dresidual"], "norm_weight": an["dweight"], "head_weight": gn["dweight"],
                "decay_bias": da.sum((0, 1)), "w_in": dp.t() @ u2, "w_out": d2.t() @ o.view(B * L, -1)}


def reference(block, x, residual, weights):
    """The same block token by token in plain float32 operations."""
    n, w_in, hw, w_out, bias = weights
    B, L, _ = x.shape
    H, G, d = block.H, block.G, block.d
    r = residual + x
    u = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + 1e-5) * n
    q, k, v, z, a = (u @ w_in.t())[..., :sum(block.sizes)].split(block.sizes, -1)
    q, k = (t.unflatten(-1, (G, d)).repeat_interleave(H // G, -2) for t in (q, k))
    v, decay = v.unflatten(-1, (H, d)), torch.exp(-F.softplus(a + bias))
    S, ys = x.new_zeros(B, H, d, d), []
    for t in range(L):
        S = decay[:, t, :, None, None] * S + v[:, t, :, :, None] * k[:, t, :, None, :]
        ys.append((S * q[:, t, :, None, :]).sum(-1) * d ** -0.5)
    y = torch.stack(ys, 1)
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-5) * hw.view(H, d)
    return (y.flatten(2) * F.silu(z)) @ w_out.t(), r


def check(block, L=96, steps=8, batch=2, device="cuda"):
    """Errors (of each result's largest value) of the prompt, of tokens that follow a prompt,
    and of the gradients, against plain float32."""
    D = block.norm_weight.numel()
    r = torch.Generator(device="cpu").manual_seed(1)
    x = torch.randn(batch, L, D, generator=r).to(device, BF16)
    res = torch.randn(batch, L, D, generator=r).to(device)
    dout = torch.randn(batch, L, D, generator=r).to(device, BF16)
    dres = torch.randn(batch, L, D, generator=r).to(device)
    leaves = [t.float().clone().requires_grad_() for t in (block.norm_weight, block.w_in, block.head_weight, block.w_out, block.decay_bias)]
    xf, rf = x.float().requires_grad_(), res.clone().requires_grad_()
    want, want_r = reference(block, xf, rf, leaves)
    (want * dout.float() + want_r * dres).sum().backward()

    def err(got, ref):
        return ((got.float() - ref).abs().max() / ref.abs().max()).item()

    out, new, _ = block.prompt(x, res)
    errors = {"prompt": err(out, want.detach()), "residual": err(new, want_r.detach())}
    cut = L - steps
    _, _, state = block.prompt(x[:, :cut].contiguous(), res[:, :cut].contiguous())
    toks = [block.token(x[:, t].contiguous(), res[:, t].contiguous(), state)[0] for t in range(cut, L)]
    errors["tokens"] = err(torch.stack(toks, 1), want.detach()[:, cut:])
    g = block.gradients(x, res, dout, dres)
    for name, leaf in zip(("norm_weight", "w_in", "head_weight", "w_out", "decay_bias", "x", "residual"), (*leaves, xf, rf)):
        errors["d " + name] = err(g[name], leaf.grad)
    return errors


def main():
    small = LinAttnBlock()
    for name, e in check(small).items():
        print(f"{name:14s} {e:.1e} of its largest value from plain float32")
    block = LinAttnBlock(width=2560, heads=40, groups=40, dim=64, group=128)
    x = torch.randn(1, 4096, 2560, device="cuda").to(BF16)
    res = torch.zeros(1, 4096, 2560, device="cuda")

    def timed(what, f, n):
        f()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(n):
            f()
        torch.cuda.synchronize()
        print(f"{what}: {(time.perf_counter() - t) / n * 1e6:.0f} us")

    _, _, state = block.prompt(x, res)
    timed("prompt of 4096 tokens, one block", lambda: block.prompt(x, res), 10)
    one, r1 = x[:, 0].contiguous(), res[:, 0].contiguous()
    timed("one token, one block", lambda: block.token(one, r1, state), 50)
    timed("forward and backward over 4096 tokens, one block", lambda: block.gradients(x, res, x, res), 5)


if __name__ == "__main__":
    main()
