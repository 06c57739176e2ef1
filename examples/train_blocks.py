"""Trains a stack of equivariant residual blocks on synthetic graphs.

One block is   y -> convolution -> (gates q | features z) -> post-norm, gate, residual scale and
residual, with the next block's pre-norm in the same kernel.  The convolution is the radial uvw
one; its output row holds the gates in front of the features, and the norm reads both as column
ranges and writes their gradients as column ranges of the convolution's output gradient.  A step
ends in the global gradient norm and AdamW.  Targets come from a second network with other weights.

    python examples/train_blocks.py [--steps 60] [--nodes 512] [--blocks 2] [--state 8bit]
"""

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import clebsch_gordan_tensor_racah_gb300 as cg  # noqa: E402
from clebsch_gordan_tensor_racah_gb300 import workloads as wl  # noqa: E402

MUL, K = 32, 8
IRREPS = f"{MUL}x0e+{MUL}x1o+{MUL}x2e"
SH = "0e+1o+2e"


class Blocks:
    """`count` residual blocks and a readout of the scalars, with explicit backward passes."""

    def __init__(self, count, nodes, seed):
        self.count = count
        self.norms = [cg.ResNormPlan(IRREPS, act="none")] + [cg.ResNormPlan(IRREPS, act="silu") for _ in range(count)]
        self.dim, self.chan = self.norms[0].dim, self.norms[0].channels
        out = f"{self.chan}x0e+{IRREPS}"        # gates, then features
        paths = [(i, j, o) for o, lo in enumerate((0, 0, 1, 2)) for i in range(3) for j in range(3)
                 if abs(i - j) <= lo <= i + j and (i + j + lo) % 2 == 0]
        self.convs = [cg.Plan(IRREPS, SH, out, "uvw", radial_k=K, instructions=paths) for _ in range(count)]
        for c in self.convs:
            c.set_node_chunk(nodes)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        draw = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
        self.mix = [draw(K, c.w_numel) / (K * MUL) ** 0.5 for c in self.convs]
        self.pre = [1 + 0.1 * draw(self.chan) for _ in range(count + 1)]
        self.post = [1 + 0.1 * draw(self.chan) for _ in range(count)]
        self.scale = [0.5 + 0.1 * draw(self.chan) for _ in range(count)]
        self.readout = draw(MUL) / MUL ** 0.5

    def parameters(self):
        return self.mix + self.pre + self.post + self.scale + [self.readout]

    def forward(self, graph, h, Y, R):
        """Prediction [N] and what the backward needs."""
        kept = []
        x, y = cg.cgtp_resnorm_forward(self.norms[0], h, pre=self.pre[0])
        for b in range(self.count):
            o = cg.cgtp_conv_forward(self.convs[b], graph, y, Y, R, self.mix[b])
            kept.append((x, y, o))
            q, z = o[:, :self.chan], o[:, self.chan:]
            x, y = cg.cgtp_resnorm_forward(self.norms[b + 1], x, z, q, post=self.post[b], scale=self.scale[b], pre=self.pre[b + 1])
        kept.append((x, y, None))
        return y[:, :MUL] @ self.readout, kept

    def backward(self, graph, Y, R, gpred, kept):
        """Gradients in the order of parameters()."""
        y = kept[-1][1]
        g_read = y[:, :MUL].t() @ gpred
        gy = torch.zeros_like(y)
        gy[:, :MUL] = gpred[:, None] * self.readout
        g_mix, g_pre, g_post, g_scale = [None] * self.count, [None] * (self.count + 1), [None] * self.count, [None] * self.count
        gx = None
        for b in reversed(range(self.count)):
            h, y_in, o = kept[b]
            x = kept[b + 1][0]
            q, z, go = o[:, :self.chan], o[:, self.chan:], torch.empty_like(o)
            gh = torch.empty_like(h)
            sums = [torch.empty(self.chan, device="cuda") for _ in range(3)]
            cg.cgtp_resnorm_backward(self.norms[b + 1], gx, gy, x, z, q, post=self.post[b], scale=self.scale[b], pre=self.pre[b + 1],
                                     outs=(gh, go[:, self.chan:], go[:, :self.chan], *sums))
            g_post[b], g_scale[b], g_pre[b + 1] = sums
            gy, _, _, g_mix[b] = cg.cgtp_conv_backward(self.convs[b], graph, go, y_in, Y, R, self.mix[b])
            gx = gh
        *_, g_pre[0] = cg.cgtp_resnorm_backward(self.norms[0], gx, gy, kept[0][0], pre=self.pre[0], need_gh=False)
        return g_mix + g_pre + g_post + g_scale + [g_read]


def train(steps=60, nodes=512, blocks=2, state="f32", seed=0, degree=16, report=print):
    """Losses of `steps` AdamW steps."""
    rng = np.random.default_rng(seed)
    rowptr, col = wl.graph_fixed_indegree(rng, nodes, degree)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    graph = cg.Graph(dev(rowptr), dev(col), nodes)
    edges = nodes * degree
    Y = dev(wl.sh_real(2, wl.unit_vectors(rng, edges)).astype(np.float32))
    R = dev((wl.rbf(rng.uniform(0.5, 5.0, edges), K) / degree ** 0.5).astype(np.float32))
    teacher, net = Blocks(blocks, nodes, seed + 1), Blocks(blocks, nodes, seed + 2)
    h = torch.zeros(nodes, net.dim, device="cuda")
    h[:, :MUL] = dev(rng.standard_normal((nodes, MUL)).astype(np.float32))     # node types: scalars only
    target, _ = teacher.forward(graph, h, Y, R)
    params = net.parameters()
    # gains, scales and the readout are not decayed
    opt = cg.AdamW([p.numel() for p in params], state=state, decay_scale=[1.0 if p.dim() > 1 else 0.0 for p in params])
    moments = opt.new_state()
    losses = []
    for t in range(1, steps + 1):
        pred, kept = net.forward(graph, h, Y, R)
        off = pred - target
        losses.append((off * off).mean())
        grads = net.backward(graph, Y, R, 2 * off / nodes, kept)
        clip = cg.cgtp_grad_norm(opt, grads, max_norm=10.0)
        cg.cgtp_adamw_step(opt, params, grads, moments, lr=5e-3, weight_decay=1e-4, step=t, clip=clip, seed=seed)
        if report and (t == 1 or t % 20 == 0):
            report(f"step {t:4d}  loss {float(losses[-1]):.5f}  gradient norm {float(clip[0]):.4f}")
    return [float(v) for v in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--nodes", type=int, default=512)
    ap.add_argument("--blocks", type=int, default=2)
    ap.add_argument("--state", choices=("f32", "8bit"), default="f32")
    a = ap.parse_args()
    train(a.steps, a.nodes, a.blocks, a.state)
