"""A feed-forward layer, dense or of experts, around a residual stream: a prompt,
token-by-token steps (from the host, then from a captured graph) and a training
step with the routers' balance term.

A dense layer is

    u      = norm(stream)                            rms_norm_fwd
    h      = silu(u W1g^T) * (u W1u^T)               linear_fwd, "swiglu"
    stream = stream + h W2^T                         linear_fwd, residual in place

and a layer of experts, each token's rows through the k experts it is sent to,

    p, e   = top k of softmax(u Wr^T)                linear_fwd, expert_route_fwd
    order  = rows by expert                          expert_sort
    h      = swiglu(u W1[e]^T), y = h W2[e]^T        expert_linear_fwd
    stream = stream + sum over k of p y              expert_combine_fwd, in place

    python examples/expert_layer.py [--dim 768 --hidden 768 --experts 16 ...]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import selective_state_space_38_amd as ssm  # noqa: E402

ACT = "swiglu"


class Dense:
    """Parameters of a dense layer, drawn from a seed (random, not trained)."""

    def __init__(self, dim, hidden, seed, dtype=torch.bfloat16, device="cuda"):
        gen = torch.Generator().manual_seed(seed)
        self.norm = torch.ones(dim, device=device)
        self.w1 = (torch.randn(2 * hidden, dim, generator=gen) * dim ** -0.5).to(device, dtype)
        self.w2 = (torch.randn(dim, hidden, generator=gen) * hidden ** -0.5).to(device, dtype)

    def params(self):
        return [self.norm, self.w1, self.w2]

    def step(self, u, stream):
        h = ssm.linear_fwd(u, self.w1, activation=ACT)
        return ssm.linear_fwd(h, self.w2, residual=stream, out=stream)

    def train(self, u, stream):
        return stream + Linear.apply(Linear.apply(u, self.w1, ACT), self.w2, None), 0.0


class Experts:
    """Parameters of a layer of experts."""

    def __init__(self, dim, hidden, experts, k, seed, dtype=torch.bfloat16, device="cuda"):
        gen = torch.Generator().manual_seed(seed)

        def normal(*shape):
            return (torch.randn(*shape, generator=gen) * shape[-1] ** -0.5).to(device, dtype)

        self.k, self.experts = k, experts
        self.norm = torch.ones(dim, device=device)
        self.wr, self.w1, self.w2 = normal(experts, dim), normal(experts, 2 * hidden, dim), \
            normal(experts, dim, hidden)

    def params(self):
        return [self.norm, self.wr, self.w1, self.w2]

    def step(self, u, stream):
        logits = ssm.linear_fwd(u, self.wr, out_dtype=torch.float32)
        index, weight = ssm.expert_route_fwd(logits, self.k, renormalize=True)
        offsets, token, slot = ssm.expert_sort(index, self.experts)
        h = ssm.expert_linear_fwd(u, self.w1, offsets, token=token, activation=ACT)
        y = ssm.expert_linear_fwd(h, self.w2, offsets)
        return ssm.expert_combine_fwd(y, slot, weight, residual=stream, out=stream)

    def train(self, u, stream):
        logits = Linear.apply(u, self.wr, None)
        weight, index, total = Route.apply(logits, self.k)
        offsets, token, slot = ssm.expert_sort(index, self.experts)
        h = ExpertLinear.apply(u, self.w1, offsets, token, slot, ACT)
        y = ExpertLinear.apply(h, self.w2, offsets, None, None, None)
        # the balance term: experts that are asked for often should score less
        share = (offsets[1:] - offsets[:-1]).float() / token.numel()
        balance = self.experts * (share * total).sum() / len(u)
        return stream + Combine.apply(y, slot, weight), balance


def forward(layers, tokens):
    """tokens [T, dim] bfloat16 -> the float32 stream."""
    stream = tokens.float()
    for layer in layers:
        u = ssm.rms_norm_fwd(stream, layer.norm).to(layer.w1.dtype)
        stream = layer.step(u, stream)
    return stream


def capture(layers, tokens):
    """forward as a graph: (graph, output); a replay takes what tokens then holds."""
    forward(layers, tokens)                  # allocations outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = forward(layers, tokens)
    return graph, out


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, s, weight):
        ctx.save_for_backward(s, weight)
        return ssm.rms_norm_fwd(s, weight)

    @staticmethod
    def backward(ctx, dy):
        s, weight = ctx.saved_tensors
        g = ssm.rms_norm_bwd(dy.contiguous(), s, weight)
        return g["ds"], g["dweight"]


class Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, act):
        out, pre = ssm.linear_fwd(x, w, activation=act, return_pre=True)
        ctx.act = act
        ctx.save_for_backward(x, w, pre if act else None)
        return out

    @staticmethod
    def backward(ctx, dout):
        x, w, pre = ctx.saved_tensors
        g = ssm.linear_bwd(dout.contiguous(), x, w, activation=ctx.act, pre=pre)
        return g["dx"], g["dw"], None


class Route(torch.autograd.Function):
    """logits -> weight, index, score_sum; the weights and the sum have gradients."""

    @staticmethod
    def forward(ctx, logits, k):
        index, weight, total = ssm.expert_route_fwd(logits, k, renormalize=True,
                                                    return_score_sum=True)
        ctx.save_for_backward(logits, index)
        ctx.mark_non_differentiable(index)
        return weight, index, total

    @staticmethod
    def backward(ctx, dweight, _, dtotal):
        logits, index = ctx.saved_tensors
        return ssm.expert_route_bwd(logits, index, dweight.contiguous(), renormalize=True,
                                    dscore_sum=dtotal.contiguous()), None


class ExpertLinear(torch.autograd.Function):
    """Rows by expert; with token, x holds the tokens and its gradient is summed by token."""

    @staticmethod
    def forward(ctx, x, w, offsets, token, slot, act):
        out, pre = ssm.expert_linear_fwd(x, w, offsets, token=token, activation=act,
                                         return_pre=True)
        ctx.act = act
        ctx.save_for_backward(x, w, offsets, token, slot, pre if act else None)
        return out

    @staticmethod
    def backward(ctx, dout):
        x, w, offsets, token, slot, pre = ctx.saved_tensors
        g = ssm.expert_linear_bwd(dout.contiguous(), x, w, offsets, token=token,
                                  activation=ctx.act, pre=pre)
        dx = g["dx"] if slot is None else ssm.expert_combine_fwd(g["dx"], slot)
        return dx, g["dw"], None, None, None, None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, slot, weight):
        ctx.save_for_backward(y, slot, weight)
        return ssm.expert_combine_fwd(y, slot, weight)

    @staticmethod
    def backward(ctx, dout):
        y, slot, weight = ctx.saved_tensors
        g = ssm.expert_combine_bwd(dout.contiguous(), y, slot, weight)
        return g["dy"], None, g["dweight"]


def loss_of(layers, tokens, target, balance_rate=1e-2):
    stream, balance = tokens.float(), 0.0
    for layer in layers:
        u = Norm.apply(stream, layer.norm).to(layer.w1.dtype)
        stream, more = layer.train(u, stream)
        balance = balance + more
    return (stream - target).square().mean() + balance_rate * balance


def train(layers, tokens, target, steps, rate=1e-2):
    """Plain gradient descent; returns the losses."""
    params = [p.requires_grad_() for layer in layers for p in layer.params()]
    losses = []
    for _ in range(steps):
        loss = loss_of(layers, tokens, target)
        grads = torch.autograd.grad(loss, params)
        with torch.no_grad():
            for p, g in zip(params, grads):  # steps in proportion to the parameter
                g = g.float()
                p -= (rate * g / (g.square().mean().sqrt() + 1e-12) * p.float().abs().mean()).to(p.dtype)
        losses.append(loss.detach())
    for p in params:
        p.requires_grad_(False)
    return [float(v) for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--dim", type=int, default=768)
    ap.add_argument("--hidden", type=int, default=768)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--k", type=int, default=4)
    ap.add_argument("--layers", type=int, default=4, help="dense and of experts in turn")
    ap.add_argument("--tokens", type=int, default=8192)
    ap.add_argument("--batch", type=int, default=8, help="tokens of a decode step")
    ap.add_argument("--steps", type=int, default=64, help="decode steps")
    ap.add_argument("--train-steps", type=int, default=10)
    args = ap.parse_args()
    layers = [Experts(args.dim, args.hidden, args.experts, args.k, i) if i % 2 else
              Dense(args.dim, args.k * args.hidden, i) for i in range(args.layers)]
    gen = torch.Generator().manual_seed(0)
    tokens = torch.randn(args.tokens, args.dim, generator=gen).bfloat16().cuda()

    losses = train(layers, tokens, tokens.float().roll(1, 0) * 0.5, args.train_steps)
    print(f"training: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {args.train_steps} steps")

    def timed(f, n):
        f()
        torch.cuda.synchronize()
        start = time.perf_counter()
        for _ in range(n):
            f()
        torch.cuda.synchronize()
        return (time.perf_counter() - start) / n

    print(f"prompt: {args.tokens} tokens in {timed(lambda: forward(layers, tokens), 3) * 1e3:.2f} ms")
    few = tokens[:args.batch].clone()
    print(f"decode: {timed(lambda: forward(layers, few), args.steps) * 1e6:.0f} us a step of "
          f"{args.batch} tokens")
    graph, _ = capture(layers, few)
    print(f"decode from a graph: {timed(graph.replay, args.steps) * 1e6:.0f} us a step")


if __name__ == "__main__":
    main()
