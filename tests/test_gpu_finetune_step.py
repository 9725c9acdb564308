"""The operators together, as a training step of adapters beside the frozen
layer uses them: adapters of the router's projection -> routing and the layer ->
adapters of the layer's output in place; the balance loss of the routing, its
gradient into the router's adapters, and the output's gradient into both."""
import numpy as np
import pytest
import torch

import int4_weight_only_moe_amd as moe
import oracle
import workloads as wl
from gpu_common import assert_output_close, device_layer, oracle_experts, to_dev, x_device
from test_gpu_lora import bf16, roundings, within

pytestmark = pytest.mark.gpu

SHAPE = wl.LayerShape(E=64, H=1024, I=384, k=6)
SEQ = (0, 20, 20, 61)  # three packed sequences (one empty) and three rows of padding


class Step:
    def __init__(self, M):
        s, rng = SHAPE, np.random.default_rng(M)
        self.M, self.L, self.rr, self.ro = M, 3, 8, 16
        t = wl.tokens(s, M, 70)
        self.logits0, self.x_bits = t.logits, t.x_bits
        self.layer = device_layer(s, 3)
        ids = rng.integers(-1, self.L, M).astype(np.int32)
        self.ids = ids
        self.ar, self.br = bf16(rng.standard_normal((3, 8, s.H)) * s.H ** -0.5), bf16(rng.standard_normal((3, s.E, 8)))
        self.ao, self.bo = bf16(rng.standard_normal((3, 16, s.H)) * s.H ** -0.5), bf16(rng.standard_normal((3, s.H, 16)))
        self.sr = torch.tensor([0.5, 1.0, 2.0])
        self.so = torch.tensor([1.0, 0.25, 0.5])
        self.dy = bf16(rng.standard_normal((M, s.H)) * 0.1)
        self.gl = torch.tensor([0.01, 0.01, 0.01])
        self.d = {n: getattr(self, n).cuda() for n in ("ar", "br", "ao", "bo", "sr", "so", "dy", "gl")}
        self.d.update(x=x_device(self.x_bits), logits0=to_dev(self.logits0), ids=torch.from_numpy(ids).cuda(),
                      seq=torch.tensor(SEQ, dtype=torch.int32, device="cuda"))
        self.rb = moe.alloc_route_buffers(M, s.E, s.k, moe.moe_w4a16_preferred_block_m(M, s.E, s.H, s.I, s.k))
        self.bal = moe.alloc_balance_buffers(M, s.E, 3)
        self.hr, self.ho = torch.zeros((M, 8), device="cuda"), torch.zeros((M, 16), device="cuda")
        self.dlogits = torch.zeros((M, s.E), device="cuda")  # the padding's rows stay zero

    def run(self):
        d, s = self.d, SHAPE
        self.logits = moe.lora_forward(d["x"], d["ids"], d["ar"], d["br"], d["sr"], base=d["logits0"], h=self.hr)
        self.out = moe.layer(self.logits, d["x"], self.rb, s.I, self.layer.w13, self.layer.w2)
        self.layer_out = self.out.clone()
        moe.lora_forward(d["x"], d["ids"], d["ao"], d["bo"], d["so"], base=self.out, out=self.out, h=self.ho)
        moe.balance_loss(self.logits, self.rb.topk_ids, self.bal, seq_offsets=d["seq"])
        moe.balance_loss_backward(self.logits, s.k, self.bal.expert_counts, self.bal.seq_tokens, d["gl"],
                                  seq_offsets=d["seq"], grad_logits=self.dlogits)
        self.router = moe.lora_backward(self.dlogits, d["x"], d["ids"], self.hr, d["ar"], d["br"], d["sr"])
        self.output = moe.lora_backward(d["dy"], d["x"], d["ids"], self.ho, d["ao"], d["bo"], d["so"],
                                        dx_base=self.router[0])


def test_adapter_training_step():
    M = 64
    st = Step(M)
    st.run()
    torch.cuda.synchronize()
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    x = wl.f32_from_bf16_bits(st.x_bits).astype(np.float64)
    H, E = SHAPE.H, SHAPE.E

    # router's adapters: bounds as in test_gpu_lora (h's sum, the expansion's sum, the result's rounding)
    want, h = oracle.lora_forward(x, st.ids, f64(st.ar), f64(st.br), st.sr.numpy(), st.logits0)
    mag, hmag = oracle.lora_forward(np.abs(x), st.ids, np.abs(f64(st.ar)), np.abs(f64(st.br)), st.sr.numpy(),
                                    np.zeros((M, E)))
    within(st.logits, want, mag * (roundings(H) + roundings(8, 3) + 2.0 ** -24) + 2.0 ** -23 * np.abs(want), "logits")
    within(st.hr, h, hmag * roundings(H), "h")

    # the layer on those logits, then the output's adapters in place on what it gave
    logits = st.logits.cpu().numpy()
    ids, w = oracle.route(logits, SHAPE.k)
    np.testing.assert_array_equal(st.rb.topk_ids.cpu().numpy(), ids)
    ref = oracle.moe_forward(x, ids, w, oracle_experts(SHAPE, 3))
    assert_output_close(st.layer_out.float().cpu().numpy(), ref, "layer")
    want, _ = oracle.lora_forward(x, st.ids, f64(st.ao), f64(st.bo), st.so.numpy(), f64(st.layer_out))
    mag, _ = oracle.lora_forward(np.abs(x), st.ids, np.abs(f64(st.ao)), np.abs(f64(st.bo)), st.so.numpy(),
                                 np.zeros((M, H)))
    err = mag * (roundings(H) + roundings(16, 2) + 2.0 ** -17)
    within(st.out, want, err + 2.0 ** -8 * (np.abs(want) + err) + 2.0 ** -23 * np.abs(f64(st.layer_out)), "out")

    # balance of the routing that the layer used
    bal = oracle.balance(logits, ids, SEQ)
    np.testing.assert_array_equal(st.bal.expert_counts.cpu().numpy(), bal["counts"])
    assert st.bal.seq_tokens.tolist() == [20, 0, 41]
    np.testing.assert_allclose(st.bal.loss.cpu().numpy(), bal["loss"], rtol=60 * 2.0 ** -24)
    dl = oracle.balance_backward(logits, SHAPE.k, bal["counts"], bal["tokens"], st.gl.numpy(), SEQ)
    got = f64(st.dlogits)
    assert (got[61:] == 0).all()
    scale = np.abs(dl[:61]).max()
    assert np.abs(got[:61] - dl[:61]).max() <= 200 * 2.0 ** -24 * scale * E  # c - sum c p cancels: up to E-fold terms

    # gradients of both adapters from what the device had
    for name, grads, dout, hh, a, b, s, base in (
            ("router", st.router, got, f64(st.hr), st.ar, st.br, st.sr, np.zeros((M, H))),
            ("output", st.output, f64(st.dy), f64(st.ho), st.ao, st.bo, st.so, f64(st.router[0]))):
        s = s.numpy()
        args = (dout, x, st.ids, hh, f64(a), f64(b), s)
        dx, da, db = oracle.lora_backward(*args, base)
        mdx, mda, mdb = oracle.lora_backward(*(np.abs(v) if i != 2 else v for i, v in enumerate(args)), np.zeros((M, H)))
        dh = roundings(dout.shape[1], 3) + 2.0 ** -24
        err = mdx * (dh + roundings(16, 2) + 2.0 ** -17)
        within(grads[0], dx, err + 2.0 ** -8 * (np.abs(dx) + err) + 2.0 ** -23 * np.abs(base), name + " dx")
        within(grads[1], da, mda * (dh + roundings(M, 3) + 2.0 ** -23), name + " da")
        within(grads[2], db, mdb * (roundings(M, 6) + 2.0 ** -22), name + " db")


def test_adapter_training_step_in_a_graph():
    """Captured once and replayed on other inputs; the eager step on those inputs gives the same bits
    (of what does not go through the layer's atomic sums)."""
    M = 64
    st = Step(M)
    st.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st.run()
    captured = (st.logits, st.dlogits, st.bal.loss, st.router, st.ho)
    for rep in range(4):
        rng = np.random.default_rng(rep)
        st.d["ids"].copy_(torch.from_numpy(rng.integers(-1, 3, M).astype(np.int32)).cuda())
        st.d["x"].copy_(bf16(rng.standard_normal((M, SHAPE.H))).cuda())
        for t in (st.dlogits, st.bal.loss, st.bal.workspace, st.hr, st.ho):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (captured[0], captured[1], captured[2], *captured[3], captured[4])]
        st.run()
        torch.cuda.synchronize()
        want = (st.logits, st.dlogits, st.bal.loss, *st.router, st.ho)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), rep
        assert torch.isfinite(st.output[0].float()).all()
