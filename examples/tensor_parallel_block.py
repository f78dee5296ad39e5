"""A tensor-parallel feed-forward block, forward and backward, on one GPU.

Every rank holds a slice of the two weights. A rank's part is
    u = gelu(y w1^T + b1),  partial = u w2^T
and the partials are summed over the ranks by the one-shot all-reduce; then
    h = x + dropout(sum + b2),  out = layer_norm(h)
on every rank alike, with the same mask, which nothing stores. Backward, the
gradient of the block's input is a partial sum again and takes the all-reduce.

This GPU is rank 0. The peers are virtual: their partials are computed here
too, with their own slices, and put into the recv slots that a peer would
write (arx.h, arx_allreduce).

    python examples/tensor_parallel_block.py [tokens [hidden [inner [world]]]]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from signal_pad_sync_amd import arx  # noqa: E402

BF16 = torch.bfloat16


class Block:
    """Weights of all ranks, and one rank's calls."""

    def __init__(self, hidden, inner, world, p=0.1, seed=1):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale=1.0, shift=0.0):
            return (torch.randn(*shape, generator=g, device="cuda") * scale + shift).to(BF16)
        share = inner // world
        self.world, self.p, self.seed = world, p, seed
        self.w1 = [normal(share, hidden, scale=hidden ** -0.5) for _ in range(world)]
        self.b1 = [normal(share, scale=0.1) for _ in range(world)]
        self.w2 = [normal(hidden, share, scale=inner ** -0.5) for _ in range(world)]
        self.b2, self.weight, self.shift = normal(hidden, scale=0.1), normal(hidden, scale=0.1, shift=1.0), normal(
            hidden, scale=0.1)
        self.calls = 0

    def all_reduce(self, partials):
        """Sum over the ranks; every rank but this one has put its partial into
        this call's slot."""
        self.calls += 1
        n = partials[0].numel()
        for src in range(1, self.world):
            arx.recv_view(self.calls & 1, src, n).copy_(partials[src].reshape(-1))
        out = torch.empty_like(partials[0])
        arx.allreduce(partials[0], out, n)
        return out

    def forward(self, x, y, step):
        """x: the residual stream, y: its norm. Returns what the next block takes
        (h, out) and what the backward pass needs."""
        kept, partials = [], []
        for r in range(self.world):   # rank r's own calls
            u, z = arx.linear(y, self.w1[r], bias=self.b1[r], act="gelu", save_z=True)
            partials.append(arx.linear(u, self.w2[r]))
            kept.append((u, z))
        total = self.all_reduce(partials)
        h, out, mean, rstd = arx.dropout_add_norm(total, x, self.weight, self.shift, bias=self.b2, p=self.p,
                                                  seed=self.seed, offset=step)
        return h, out, (y, kept, h, mean, rstd, step)

    def backward(self, dout, dh, saved):
        """Gradients from those of out and h: of x and y, and of the weights
        (rank 0's slices)."""
        y, kept, h, mean, rstd, step = saved
        dtotal, dx, db2, dweight, dshift = arx.dropout_add_norm_backward(
            dout, dh, h, mean, rstd, self.weight, p=self.p, seed=self.seed, offset=step, dbias=True)
        partials = []
        for r in range(self.world):
            u, z = kept[r]
            du, dw2, _ = arx.linear_backward(dtotal, u, self.w2[r])
            dy, dw1, db1 = arx.linear_backward(du, y, self.w1[r], z=z, act="gelu", dbias=True)
            partials.append(dy)
            if r == 0:
                grads = {"w1": dw1, "b1": db1, "w2": dw2}
        grads.update(b2=db2, weight=dweight, shift=dshift)
        return dx, self.all_reduce(partials), grads


def plain(block, x, y, dout, dh, mask):
    """The same in torch's binary32 autograd, for comparison; mask: the kept
    elements' scale."""
    f = {k: [t.float().requires_grad_() for t in getattr(block, k)] for k in ("w1", "b1", "w2")}
    v = {k: getattr(block, k).float().requires_grad_() for k in ("b2", "weight", "shift")}
    x, y = x.float().requires_grad_(), y.float().requires_grad_()
    total = sum(torch.nn.functional.gelu(y @ f["w1"][r].t() + f["b1"][r]) @ f["w2"][r].t() for r in range(block.world))
    h = x + (total + v["b2"]) * mask
    out = torch.nn.functional.layer_norm(h, h.shape[1:], v["weight"], v["shift"])
    ((out * dout.float()).sum() + (h * dh.float()).sum()).backward()
    want = {"h": h, "out": out, "dx": x.grad, "dy": y.grad}
    want.update({k: f[k][0].grad for k in f})
    want.update({k: v[k].grad for k in v})
    return want


def run(tokens=256, hidden=4096, inner=16384, world=8, p=0.1):
    """One step of the block and the plain form; relative errors (2-norm) by name."""
    g = torch.Generator(device="cuda").manual_seed(7)
    x, dout, dh = ((torch.randn(tokens, hidden, generator=g, device="cuda") * s).to(BF16) for s in (1.0, 0.1, 0.1))
    arx.init(world, tokens * hidden)
    try:
        block = Block(hidden, inner, world, p)
        y = arx.layer_norm(x, block.weight, block.shift)[0]
        h, out, saved = block.forward(x, y, step=3)
        dx, dy, grads = block.backward(dout, dh, saved)
        torch.cuda.synchronize()
    finally:
        arx.finalize()
    ones = torch.ones(tokens, hidden, device="cuda")
    mask = arx.dropout_add(ones, p=p, seed=block.seed, offset=3)
    want = plain(block, x, y, dout, dh, mask)
    got = {"h": h, "out": out, "dx": dx, "dy": dy, **grads}
    return {k: float((got[k].float() - want[k].detach()).norm() / want[k].detach().norm()) for k in want}


if __name__ == "__main__":
    errors = run(*(int(v) for v in sys.argv[1:5]))
    for name, e in errors.items():
        print(f"{name:8s} relative error {e:.2e}")
    # values pass through at most about eight roundings to bf16 of 2^-8 each
    assert max(errors.values()) < 8 * 2.0 ** -8, errors
    print("tensor-parallel block ok")
