"""The operators together, as a model uses them around the layer: the norm that
takes the last sublayer's output into the residual stream, the router's
projection (torch's product), routing by scores, the layer, the next norm with the
layer's output; and a training step of the router and the norms: gradients of the
routing's weights and of the balance loss by the logits, of the norms, clipped
together."""
import numpy as np
import pytest
import torch

import int4_weight_only_moe_amd as moe
import oracle
import workloads as wl
from gpu_common import assert_output_close, device_layer, oracle_experts

pytestmark = pytest.mark.gpu

SHAPE = wl.LayerShape(E=32, H=512, I=256, k=4)
GROUPS = (4, 2, 2)
BF16 = torch.bfloat16


class Block:
    """Buffers and weights of one block for M tokens; run() allocates nothing of the package's."""

    def __init__(self, M, stream, seed=1):
        s, g = SHAPE, torch.Generator().manual_seed(seed)
        self.M, self.layer = M, device_layer(s, 3)
        normal = lambda *shape, scale=1.0: (scale * torch.randn(*shape, generator=g)).cuda()  # noqa: E731
        self.residual0 = normal(M, s.H, scale=3.0).to(stream)
        self.delta = normal(M, s.H).to(BF16)
        self.w1, self.w2 = ((1 + normal(s.H, scale=0.2)).to(BF16) for _ in range(2))
        self.router = normal(s.E, s.H, scale=s.H ** -0.5)
        self.bias = normal(s.E, scale=0.05)
        self.valid = torch.ones(M, dtype=torch.bool, device="cuda")
        self.valid[M // 2:M // 2 + M // 5] = False
        self.n1 = moe.alloc_norm_buffers(M, s.H, stream, rstd=True)
        self.n2 = moe.alloc_norm_buffers(M, s.H, stream, rstd=True, quant_group=128)
        self.rb = moe.alloc_route_buffers(M, s.E, s.k, moe.moe_w4a16_preferred_block_m(M, s.E, s.H, s.I, s.k))
        self.bal = moe.alloc_balance_buffers(M, s.E)
        self.ws = torch.empty(max(moe.moe_w4a16_workspace_bytes(M, s.E, s.H, s.I, s.k), 16), dtype=torch.uint8, device="cuda")
        self.out = torch.empty((M, s.H), dtype=BF16, device="cuda")
        # what comes back from the rest of the model
        self.dy, self.dh = normal(M, s.H, scale=0.1).to(BF16), normal(M, s.H, scale=0.1).to(stream)
        self.dweights = normal(M, s.k, scale=0.1)
        self.gl = torch.full((1,), 0.01, device="cuda")
        self.dlogits = torch.zeros((M, s.E), device="cuda")
        self.norm_ws = torch.empty(moe.moe_add_rms_norm_workspace_bytes(M, s.H), dtype=torch.uint8, device="cuda")
        like = lambda t: (torch.empty((M, s.H), dtype=stream, device="cuda"), torch.empty(s.H, device="cuda"))  # noqa: E731
        self.g1, self.g2 = like(0), like(0)
        self.drouter = torch.empty((s.E, s.H), device="cuda")
        self.clip_ws = torch.empty(moe.moe_grad_norm_workspace_bytes(3), dtype=torch.uint8, device="cuda")
        self.sumsq, self.norm = torch.empty(1, dtype=torch.float64, device="cuda"), torch.empty(1, device="cuda")
        self.clipped = [torch.empty_like(t) for t in (self.drouter, self.g1[1], self.g2[1])]

    def forward(self):
        s = SHAPE
        moe.add_rms_norm(self.delta, self.w1, self.n1, residual=self.residual0)
        self.logits = self.n1.out.float() @ self.router.t()
        moe.route_scored(self.logits, self.rb, "sigmoid", self.bias, *GROUPS, scale=2.5, row_valid=self.valid)
        moe.forward(self.n1.out, self.rb, s.I, self.layer.w13, self.layer.w2, workspace=self.ws, out=self.out)
        moe.add_rms_norm(self.out, self.w2, self.n2, residual=self.n1.residual_out)

    def backward(self):
        s = SHAPE
        moe.add_rms_norm_backward(self.dy, self.n2.residual_out, self.n2.rstd, self.w2, grad_residual=self.dh, grads=self.g2,
                                  workspace=self.norm_ws)
        moe.balance_loss(self.logits, self.rb.topk_ids, self.bal, row_valid=self.valid)
        moe.balance_loss_backward(self.logits, s.k, self.bal.expert_counts, self.bal.seq_tokens, self.gl,
                                  row_valid=self.valid, grad_logits=self.dlogits)
        moe.route_scored_backward(self.logits, self.rb.topk_ids, self.dweights, "sigmoid", scale=2.5,
                                  grad_base=self.dlogits, grad_logits=self.dlogits)
        dx = (self.dlogits @ self.router).to(BF16)
        torch.mm(self.dlogits.t(), self.n1.out.float(), out=self.drouter)
        moe.add_rms_norm_backward(dx, self.n1.residual_out, self.n1.rstd, self.w1, grad_residual=self.g2[0], grads=self.g1,
                                  workspace=self.norm_ws)
        grads = [self.drouter, self.g1[1], self.g2[1]]
        moe.grad_sumsq(grads, sumsq=self.sumsq, workspace=self.clip_ws)
        moe.grad_clip(grads, self.sumsq, 0.5, out=self.clipped, norm=self.norm)

    def results(self):
        return [self.n1.residual_out, self.n1.out, self.rb.topk_ids, self.rb.topk_weights, self.rb.sorted_token_ids,
                self.n2.residual_out, self.n2.out, self.n2.scales, self.n2.out8.view(torch.uint8), self.dlogits, *self.g1,
                *self.g2, *self.clipped, self.norm]


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("M", (1, 7, 300))
@pytest.mark.parametrize("stream", (BF16, torch.float32))
def test_block_forward(M, stream):
    s, b = SHAPE, Block(M, stream)
    b.forward()
    torch.cuda.synchronize()
    # each stage from the stage before it as the device has it
    h1 = (b.residual0.float() + b.delta.float()).to(stream)
    assert torch.equal(b.n1.residual_out, h1)
    ids, w = oracle.route_scored(b.logits.cpu().numpy(), s.k, "sigmoid", b.bias.cpu().numpy(), *GROUPS, True, 2.5,
                                 b.valid.cpu().numpy())
    np.testing.assert_array_equal(b.rb.topk_ids.cpu().numpy(), ids)
    cache = oracle_experts(s, 3)
    want = np.zeros((M, s.H))
    live = b.valid.cpu().numpy()
    want[live] = oracle.moe_forward(f64(b.n1.out)[live], ids[live], w[live], cache)
    out = b.out.float().cpu().numpy()
    assert not out[~live].any()
    assert_output_close(out, want)
    h2 = (h1.float() + b.out.float()).to(stream)
    assert torch.equal(b.n2.residual_out, h2)
    y, _ = oracle.rms_norm(f64(h2), f64(b.w2), 1e-6)
    assert (np.abs(f64(b.n2.out) - y) <= (2.0 ** -8 + 4 * 2.0 ** -24) * np.abs(y)).all()
    q, scales = oracle.quantise(y, 128)
    np.testing.assert_array_equal(b.n2.scales.cpu().numpy(), scales)
    np.testing.assert_array_equal(b.n2.out8.float().cpu().numpy(), q.astype(np.float32))


def test_block_training_step():
    """Gradients of the whole step against float64 autograd of the same function
    (the layer's output enters as a constant), each within the roundings of its
    inputs: dx is rounded to bf16 (2^-8 of each element) before the first norm's
    backward, the products are torch's in fp32."""
    M, s = 200, SHAPE
    b = Block(M, torch.float32)
    b.forward()
    b.backward()
    torch.cuda.synchronize()
    d = lambda t: t.detach().double().cpu()  # noqa: E731
    h1 = d(b.n1.residual_out)
    x = d(b.n1.out)
    router = d(b.router).requires_grad_()
    xin = x.clone().requires_grad_()
    ids, live = b.rb.topk_ids.cpu().long(), b.valid.cpu()
    logits = xin @ router.t()
    sc = torch.sigmoid(logits).gather(1, ids.clamp(min=0))
    w = 2.5 * sc / (sc.sum(1, keepdim=True) + 1e-20)
    p = torch.softmax(logits, 1) * live[:, None]
    counts = torch.zeros(s.E, dtype=torch.float64)
    counts.scatter_add_(0, ids[live].reshape(-1), torch.ones(int(live.sum()) * s.k, dtype=torch.float64))
    T = float(live.sum())
    loss = (w * d(b.dweights))[live].sum() + 0.01 * s.E / (s.k * T * T) * (counts * p.sum(0)).sum()
    loss.backward()
    np.testing.assert_allclose(f64(b.drouter), router.grad.numpy(), rtol=0, atol=1e-4 * router.grad.abs().max())

    def norm_grad(h, wt, dy, dh):
        h, wt = h.clone().requires_grad_(), d(wt).requires_grad_()
        n = h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6)
        ((n * wt * dy).sum() + (h * dh).sum()).backward()
        return h.grad, wt.grad

    g2 = norm_grad(d(b.n2.residual_out), b.w2, d(b.dy), d(b.dh))
    g1 = norm_grad(h1, b.w1, xin.grad, g2[0])
    for got, want in ((b.g2[0], g2[0]), (b.g2[1], g2[1])):
        assert (d(got) - want).abs().max() <= 1e-5 * want.abs().max()  # fp32 throughout: 70 roundings of 2^-24 are 4e-6
    # dx in bf16: half a step of each element, at most 2^-8 of the largest, through a map of norm r |w|
    for got, want in ((b.g1[0], g1[0]), (b.g1[1], g1[1])):
        assert (d(got) - want).norm() <= 2.0 ** -8 * want.norm()
    grads = [b.drouter, b.g1[1], b.g2[1]]
    root = sum(float(t.double().square().sum()) for t in grads) ** 0.5
    assert root > 0.5 and abs(b.norm.item() - root) <= 1e-6 * root
    for got, t in zip(b.clipped, grads):
        assert (d(got) - d(t) * (0.5 / root)).abs().max() <= 3e-7 * t.abs().max().item()


def test_block_step_replayed():
    """Captured whole and replayed with other inputs and the program's own work between the replays; the
    layer adds with atomics in arrival order, so what follows its output is compared within its rounding."""
    M = 150
    b = Block(M, BF16)

    def step():
        b.forward()
        b.backward()

    step()
    torch.cuda.synchronize()
    keep = b.delta.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for rep in range(4):
        b.delta.copy_(keep * (1 + rep % 3))
        for t in [*b.results(), b.norm_ws, b.clip_ws, b.ws]:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in b.results()]
        step()
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(replayed, b.results())):
            if i < 5:
                assert torch.equal(x, y), i
            elif x.is_floating_point():
                assert (x.double() - y.double()).norm() <= 0.02 * y.double().norm(), i
