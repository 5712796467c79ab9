"""A small recurrent stack on the recurrent-layer operators: trained, then served.

    python examples/recurrent_layer.py

Each block adds its input to a float32 residual stream and normalises it
(gdn_rmsnorm), projects to x, a decay gate and an input gate in one product, runs the
gated linear recurrence over the packed requests (gdn_scan, on column slices of that
product) and projects back.  With `inner` a block has a second half: norm, gated
feed-forward (gdn_glu) and projection back.  Training takes the operators' gradients
through torch.autograd.Function and clips them all together (gdn_grad_clip), by plain
descent, or as they are read by the AdamW step (gdn_adamw), whose states may be in 8 bits.  Serving
prefills a slab of states (gdn_scan) and decodes one token a request in it
(gdn_scan_step), with the norm's output in 8 bits with a scale for each 128 columns.

The task is synthetic: predict the running mean of a linear map of the inputs.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gated_delta_rule_gate_gb300 as gdn  # noqa: E402

EPS = 1e-6


class Norm(torch.autograd.Function):
    """(out, residual) of gdn_rmsnorm."""

    @staticmethod
    def forward(ctx, x, residual, weight):
        r = gdn.gdn_rmsnorm(x, weight, residual=residual, eps=EPS, want_rstd=True)
        ctx.save_for_backward(r.residual, weight, r.rstd)
        ctx.x_dtype = x.dtype
        return r.out, r.residual

    @staticmethod
    def backward(ctx, d_out, d_residual):
        residual, weight, rstd = ctx.saved_tensors
        g = gdn.gdn_rmsnorm_backward(d_out.contiguous(), residual, weight, rstd, d_residual=d_residual.contiguous())
        return g.dx.to(ctx.x_dtype), g.dx, g.dweight.to(weight.dtype)


class Scan(torch.autograd.Function):
    """gdn_scan of the three column slices of one projection; its gradients fill the
    slices of the projection's gradient."""

    @staticmethod
    def forward(ctx, xzy, bias, scale, cu):
        D = xzy.shape[1] // 3
        x, z, y = xzy.split(D, dim=1)
        out, chunks = gdn.gdn_scan(x, z, beta=y, beta_sigmoid=True, gate_bias=bias, gate_scale=scale,
                                   input_scale="unit", cu_seqlens=cu, want_chunk_states=True)
        ctx.save_for_backward(xzy, bias, scale, cu, chunks)
        return out

    @staticmethod
    def backward(ctx, d_out):
        xzy, bias, scale, cu, chunks = ctx.saved_tensors
        D = xzy.shape[1] // 3
        x, z, y = xzy.split(D, dim=1)
        d = torch.empty_like(xzy)
        dx, dz, dy = d.split(D, dim=1)
        g = gdn.gdn_scan_backward(d_out.contiguous(), x, z, chunks, beta=y, beta_sigmoid=True, gate_bias=bias,
                                  gate_scale=scale, input_scale="unit", cu_seqlens=cu, dx=dx, d_decay=dz, d_beta=dy)
        return d, g.d_gate_bias, g.d_gate_scale, None


class Glu(torch.autograd.Function):
    """gdn_glu with the gates kept for its gradient."""

    @staticmethod
    def forward(ctx, x, w_gate, w_up):
        out, gates = gdn.gdn_glu(x, w_gate, w_up, want_gates=True)
        ctx.save_for_backward(x, w_gate, w_up, gates)
        return out

    @staticmethod
    def backward(ctx, d_out):
        x, w_gate, w_up, gates = ctx.saved_tensors
        g = gdn.gdn_glu_backward(d_out.contiguous(), x, w_gate, w_up, gates, want_dx=ctx.needs_input_grad[0])
        return g.dx, g.d_w_gate, g.d_w_up


class Block:
    def __init__(self, dim, channels, gen, dtype=torch.bfloat16, device="cuda", inner=0):
        rand = lambda *s: torch.randn(*s, generator=gen, device=device)
        self.norm = torch.ones(dim, dtype=dtype, device=device)
        self.w_in = (rand(dim, 3 * channels) * dim ** -0.5).to(dtype)
        self.w_out = (rand(channels, dim) * channels ** -0.5 * 0.5).to(dtype)
        self.bias = torch.rand(channels, generator=gen, device=device) * 4 - 2
        self.log_scale = torch.rand(channels, generator=gen, device=device) * 4 - 3
        self.channels, self.inner = channels, inner
        if inner:
            self.norm2 = torch.ones(dim, dtype=dtype, device=device)
            self.w_gate, self.w_up = ((rand(inner, dim) * dim ** -0.5).to(dtype) for _ in range(2))
            self.w_down = (rand(inner, dim) * inner ** -0.5 * 0.5).to(dtype)

    def parameters(self):
        own = [self.norm, self.w_in, self.w_out, self.bias, self.log_scale]
        return own + [self.norm2, self.w_gate, self.w_up, self.w_down] if self.inner else own

    def train(self, x, residual, cu):
        y, residual = Norm.apply(x, residual, self.norm)
        out = Scan.apply(y @ self.w_in, self.bias, -torch.exp(self.log_scale), cu)
        x = out @ self.w_out
        if self.inner:
            y, residual = Norm.apply(x, residual, self.norm2)
            x = Glu.apply(y, self.w_gate, self.w_up) @ self.w_down
        return x, residual

    def serve(self, x, residual, recurrence, cu, slots, slab):
        """The same without gradients; the states of the requests are slab rows, and
        the norm hands the projection 8-bit values and scales."""
        n = gdn.gdn_rmsnorm(x, self.norm, residual=residual, eps=EPS, residual_out=residual,
                            out_dtype=torch.float8_e4m3fn, group=128)
        T, D = x.shape
        # an 8-bit product takes out and scales as they are; a plain one takes their value
        y = (n.out.float().view(T, -1, 128) * n.scales.unsqueeze(2)).view(T, D).to(x.dtype)
        x_, z, g = (y @ self.w_in).split(self.channels, dim=1)
        out = recurrence(x_, z, beta=g, beta_sigmoid=True, gate_bias=self.bias, gate_scale=-torch.exp(self.log_scale),
                         input_scale="unit", cu_seqlens=cu, slot_ids=slots, initial_state=slab, final_state=slab)
        x = out @ self.w_out
        if self.inner:
            y = gdn.gdn_rmsnorm(x, self.norm2, residual=residual, eps=EPS, residual_out=residual).out
            x = gdn.gdn_glu(y, self.w_gate, self.w_up) @ self.w_down
        return x, residual


class Stack:
    def __init__(self, blocks=2, dim=256, channels=384, seed=0, inner=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.blocks = [Block(dim, channels, gen, inner=inner) for _ in range(blocks)]
        self.dim, self.channels = dim, channels

    def parameters(self):
        return [p for b in self.blocks for p in b.parameters()]

    def train(self, x, cu):
        residual = torch.zeros(x.shape, dtype=torch.float32, device=x.device)
        for b in self.blocks:
            x, residual = b.train(x, residual, cu)
        return residual + x.float()

    def serve(self, x, recurrence, cu, slots, slabs):
        residual = torch.zeros(x.shape, dtype=torch.float32, device=x.device)
        for b, slab in zip(self.blocks, slabs):
            x, residual = b.serve(x, residual, recurrence, cu, slots, slab)
        return residual + x.float()


def offsets(lengths):
    return torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device="cuda")


def draw(lengths, dim, gen, mix):
    """Inputs, and as targets the exponential running mean (0.9) of a map of them."""
    x = torch.randn(sum(lengths), dim, generator=gen, device="cuda")
    u = x @ mix
    y, at = torch.empty_like(u), 0
    for n in lengths:
        h = torch.zeros(dim, device="cuda")
        for t in range(at, at + n):
            h = 0.9 * h + 0.1 * u[t]
            y[t] = h
        at += n
    return x.bfloat16(), 3 * y


class Descent:
    """Plain gradient descent on fp32 copies, the gradients clipped in place."""

    def __init__(self, params, rate):
        self.params, self.rate = params, rate
        self.master = [p.float() for p in params]

    def step(self, grads, max_norm):
        norm = gdn.gdn_grad_clip(grads, max_norm)
        for p, m, g in zip(self.params, self.master, grads):
            m -= self.rate * g.float()
            p.copy_(m)
        return norm


class AdamW:
    """gdn_adamw on fp32 copies of 16-bit parameters, states of `bits`; the gradients are
    clipped as they are read, and a norm that is not finite takes no step."""

    def __init__(self, params, rate, bits=32):
        self.params, self.rate, self.count = params, rate, 0
        self.master = [p.float() if p.dtype != torch.float32 else None for p in params]
        dtype = torch.float8_e4m3fn if bits == 8 else torch.float32
        self.m, self.v = ([torch.zeros(p.shape, device=p.device).to(dtype) for p in params] for _ in range(2))
        scales = lambda: [torch.zeros(-(-p.numel() // 256), device=p.device) for p in params]
        self.scales = dict(exp_avg_scales=scales(), exp_avg_sq_scales=scales()) if bits == 8 else {}

    def step(self, grads, max_norm):
        self.count += 1
        norm = gdn.gdn_grad_clip(grads, 3e38)  # measures, and leaves them as they are
        gdn.gdn_adamw(self.params, grads, self.m, self.v, self.count, lr=self.rate, master=self.master, grad_norm=norm,
                      max_norm=max_norm, **self.scales)
        return norm


def train(stack, steps=30, lengths=(100, 37, 1, 118), rate=0.5, max_norm=1.0, seed=1, optimizer=Descent):
    """Losses and gradient norms of `steps` steps."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    mix = torch.randn(stack.dim, stack.dim, generator=gen, device="cuda") * stack.dim ** -0.5
    cu = offsets(lengths)
    x, y = draw(lengths, stack.dim, gen, mix)
    params = stack.parameters()
    opt = optimizer(params, rate)
    losses, norms = [], []
    for _ in range(steps):
        for p in params:
            p.requires_grad_(True)
            p.grad = None
        loss = (stack.train(x, cu) - y).square().mean()
        loss.backward()
        grads = [p.grad for p in params]
        with torch.no_grad():
            for p in params:
                p.requires_grad_(False)
            norms.append(opt.step(grads, max_norm))
        losses.append(loss.detach())
    return [float(v) for v in losses], [float(v) for v in norms]


def serve(stack, lengths=(23, 64, 5), tokens=4, rows=8, seed=2):
    """Prefill of `lengths` and `tokens` decode steps a request in a slab of states;
    the decoded outputs, and those of one prefill over all the tokens."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B = len(lengths)
    slots = torch.randperm(rows, generator=gen, device="cuda")[:B].to(torch.int32)
    slabs = lambda: [torch.zeros(rows, stack.channels, device="cuda") for _ in stack.blocks]
    x = [torch.randn(n + tokens, stack.dim, generator=gen, device="cuda").bfloat16() for n in lengths]
    states = slabs()
    stack.serve(torch.cat([v[:n] for v, n in zip(x, lengths)]), gdn.gdn_scan, offsets(lengths), slots, states)
    one = offsets([1] * B)
    steps = [stack.serve(torch.stack([v[n + t] for v, n in zip(x, lengths)]), gdn.gdn_scan_step, one, slots, states)
             for t in range(tokens)]
    whole = [n + tokens for n in lengths]
    out = stack.serve(torch.cat(x), gdn.gdn_scan, offsets(whole), slots, slabs())
    ends = [sum(whole[:b + 1]) for b in range(B)]
    want = torch.stack([torch.stack([out[e - tokens + t] for e in ends]) for t in range(tokens)])
    return torch.stack(steps), want


def main():
    for stack, kw in ((Stack(), {}), (Stack(inner=512), dict(optimizer=AdamW, rate=3e-3)),
                      (Stack(inner=512), dict(optimizer=lambda p, rate: AdamW(p, rate, bits=8), rate=3e-3))):
        losses, norms = train(stack, **kw)
        print("loss %.4f -> %.4f, gradient norm %.3f -> %.3f" % (losses[0], losses[-1], norms[0], norms[-1]))
        got, want = serve(stack)
        print("decode against prefill: %.2g of the largest output" % float((got - want).abs().max() / want.abs().max()))


if __name__ == "__main__":
    main()
