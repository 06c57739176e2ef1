"""The training example: its explicit backward against differences of its loss, and training."""

import importlib.util
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_blocks.py")
    spec = importlib.util.spec_from_file_location("train_blocks", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_gradient_along_a_direction():
    ex = example()
    import clebsch_gordan_tensor_racah_gb300 as cg
    from clebsch_gordan_tensor_racah_gb300 import workloads as wl
    rng = np.random.default_rng(3)
    n, deg = 64, 8
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    rowptr, col = wl.graph_fixed_indegree(rng, n, deg)
    graph = cg.Graph(dev(rowptr), dev(col), n)
    Y = dev(wl.sh_real(2, wl.unit_vectors(rng, n * deg)).astype(np.float32))
    R = dev((wl.rbf(rng.uniform(0.5, 5.0, n * deg), 8) / deg ** 0.5).astype(np.float32))
    net = ex.Blocks(2, n, 7)
    h = torch.zeros(n, net.dim, device="cuda")
    h[:, :ex.MUL] = dev(rng.standard_normal((n, ex.MUL)).astype(np.float32))
    w = dev(rng.standard_normal(n).astype(np.float32))
    pred, kept = net.forward(graph, h, Y, R)
    grads = net.backward(graph, Y, R, w, kept)
    params = net.parameters()
    for i, p in enumerate(params):
        # along its own gradient, with a step of 1% of the parameter's size
        d = grads[i] / grads[i].norm()
        step = 0.01 * p.norm()
        at = []
        for s in (step, -step):
            keep = p.clone()
            p += s * d
            at.append(float((net.forward(graph, h, Y, R)[0].double() * w.double()).sum()))
            p.copy_(keep)
        slope, want = (at[0] - at[1]) / float(2 * step), float(grads[i].norm())
        # truncation: third derivative x (1%)^2 of the slope; rounding: 64 predictions of size 1 at 1e-5 (the
        # convolution's FP32 bound) over 2% of the parameter: below 3% of slopes above 0.1
        assert abs(slope - want) <= 0.03 * max(want, 0.1 / float(p.norm()) + want), (i, slope, want)


@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_training_lowers_the_loss(state):
    losses = example().train(steps=60, nodes=256, blocks=2, state=state, report=None)
    assert np.all(np.isfinite(losses))
    # the teacher has the same form: most of the variance is learned in 60 steps of 5e-3
    assert np.mean(losses[-5:]) < 0.5 * losses[0]


def test_a_step_in_a_cuda_graph():
    # the operators only enqueue kernels, so a training step can be captured and replayed
    import clebsch_gordan_tensor_racah_gb300 as cg
    torch.manual_seed(5)
    plan = cg.ResNormPlan("64x0e+64x1o", act="silu")
    n, dim, chan = 3000, plan.dim, plan.channels
    h, z, gout, gy = (torch.randn(n, dim, device="cuda") for _ in range(4))
    q, gains = torch.randn(n, chan, device="cuda"), [1 + 0.1 * torch.randn(chan, device="cuda") for _ in range(3)]
    opt = cg.AdamW([chan] * 3, state="8bit")

    def step(params, state):
        out, y = cg.cgtp_resnorm_forward(plan, h, z, q, post=params[0], scale=params[1], pre=params[2])
        grads = cg.cgtp_resnorm_backward(plan, gout, gy, out, z, q, post=params[0], scale=params[1], pre=params[2])
        clip = cg.cgtp_grad_norm(opt, list(grads[3:]), 1.0)
        cg.cgtp_adamw_step(opt, params, list(grads[3:]), state, lr=1e-2, clip=clip, seed=1)
        return out, y, grads[0], grads[1], grads[2]

    eager, captured = [g.clone() for g in gains], [g.clone() for g in gains]
    s_eager, s_captured = opt.new_state(), opt.new_state()
    for _ in range(3):
        want = step(eager, s_eager)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        got = step(captured, s_captured)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert all(torch.equal(a, b) for a, b in zip(eager, captured))
    assert all(torch.equal(s_eager[k], s_captured[k]) for k in s_eager)
