"""Routing by scores and its gradient against the float64 oracle.

Choices and grouping are bit-exact. Tolerances of weights and gradients count
roundings of 2^-24 (fp32, half a step). A sigmoid carries 2 for the
exponential, 1 for the sum and 1 for the quotient; the kept sum adds 4 steps of
joining 16 lanes to the error of its values, quotient and scale 1 each. A kept
softmax carries the difference's rounding (at most the spread of the row), 2 for
the exponential, the sum's 4, quotient and scale. A softmax over all experts is
what test_gpu_balance counts for it (twice the spread, the sum's 4 to join the
lanes and E / 16 additions rounded up to 64s, 6 for the exponential's step)."""
import itertools

import numpy as np
import pytest
import torch

import int4_weight_only_moe_amd as moe
import oracle
import workloads as wl
from gpu_common import device_layer, oracle_experts, x_device, assert_output_close

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def spread_of(logits):
    live = logits[np.isfinite(logits)]
    return float(live.max() - live.min()) if live.size else 0.0


def weight_roundings(logits, scoring, renormalise):
    E, spread = logits.shape[1], spread_of(logits)
    if scoring == "sigmoid":
        return 4 + (4 + 4 + 1 if renormalise else 0) + 1
    if renormalise:
        return 2 * (spread + 2) + 4 + 2
    return 2 * spread + 6 + 4 + 4 * (-(-E // 64)) + 2


def check_grouping(rb, ids, E):
    M, k = ids.shape
    rows, blocks, off = oracle.align_dropped(ids, E, rb.block_m)
    npp = int(rb.num_tokens_post_pad.item())
    assert npp == len(rows)
    np.testing.assert_array_equal(rb.expert_offsets.cpu().numpy(), off)
    got = rb.sorted_token_ids.cpu().numpy()
    np.testing.assert_array_equal(got[:npp], rows)
    assert (got[npp:rb.cap] == M * k).all()
    got = rb.block_expert_ids.cpu().numpy()
    np.testing.assert_array_equal(got[:len(blocks)], blocks)
    assert (got[len(blocks):rb.cap // rb.block_m] == -1).all()


def check(logits, k, scoring="softmax", bias=None, groups=(1, 1, 1), renormalise=True, scale=1.0, valid=None, block=16,
          grouping=True):
    M, E = logits.shape
    want_ids, want = oracle.route_scored(logits, k, scoring, bias, *groups, renormalise, scale, valid)
    rb = moe.alloc_route_buffers(M, E, k, block)
    for t in (rb.topk_ids, rb.sorted_token_ids, rb.block_expert_ids, rb.expert_offsets, rb.num_tokens_post_pad):
        t.fill_(77777)
    rb.topk_weights.fill_(7.0)
    moe.route_scored(dev(logits), rb, scoring=scoring, bias=dev(bias), n_groups=groups[0], top_groups=groups[1],
                     group_top=groups[2], renormalise=renormalise, scale=scale, row_valid=dev(valid), grouping=grouping)
    torch.cuda.synchronize()
    ids, w = rb.topk_ids.cpu().numpy(), rb.topk_weights.cpu().numpy()
    np.testing.assert_array_equal(ids, want_ids)
    n = weight_roundings(logits, scoring, renormalise)
    np.testing.assert_allclose(w, want, rtol=n * U, atol=2.0 ** -126)
    assert (w[want_ids < 0] == 0).all()
    if grouping:
        check_grouping(rb, want_ids, E)
    else:
        assert (rb.sorted_token_ids == 77777).all() and (rb.expert_offsets == 77777).all()
    return rb


def normal(M, E, seed):
    rng = np.random.default_rng(seed)
    return (rng.standard_normal((M, E)) + rng.standard_normal(E)).astype(np.float32)


@pytest.mark.parametrize("M,E,k,groups", [
    (1, 1, 1, (1, 1, 1)), (1, 384, 8, (1, 1, 1)), (16, 8, 2, (2, 1, 2)), (17, 60, 4, (6, 3, 2)), (33, 64, 16, (1, 1, 1)),
    (5, 100, 7, (50, 20, 2)), (64, 128, 8, (64, 8, 1)), (40, 160, 6, (8, 3, 1)), (130, 256, 8, (8, 4, 2)),
    (9, 257, 16, (257 // 257, 1, 1)), (48, 384, 8, (16, 1, 2)), (31, 512, 8, (2, 1, 2)), (20, 513, 5, (27, 9, 2)),
    (50, 1024, 16, (32, 32, 1)), (37, 1023, 11, (33, 2, 2)), (16, 1000, 16, (4, 4, 2)), (300, 7, 7, (1, 1, 1)),
    (12, 512, 16, (64, 2, 2)), (21, 62, 9, (2, 2, 2)), (19, 512, 8, (32, 4, 2)), (33, 1024, 8, (64, 5, 2)), (70, 384, 8, (24, 4, 2)),
    (15, 96, 6, (3, 2, 2)),
])
def test_route_scored_shapes(M, E, k, groups):
    logits = normal(M, E, M + E)
    rng = np.random.default_rng(E)
    for i, (scoring, biased, renormalise) in enumerate(itertools.product(("softmax", "sigmoid"), (False, True), (False, True))):
        bias = (0.1 * rng.standard_normal(E)).astype(np.float32) if biased else None
        valid = rng.random(M) > 0.2 if i % 2 else None
        lg = logits.copy()
        if valid is not None:
            lg[~valid] = np.nan
        check(lg, k, scoring, bias, groups, renormalise, 1.0 + i % 3, valid, (16, 32, 64, 128)[i % 4], grouping=i != 5)


@pytest.mark.parametrize("E,k,groups", [(65, 5, (5, 2, 2)), (100, 7, (50, 20, 2)), (128, 16, (8, 4, 2)), (160, 6, (8, 3, 1)),
                                        (256, 8, (8, 4, 2)), (257, 16, (1, 1, 1)), (384, 8, (16, 3, 2)), (384, 8, (24, 4, 2)),
                                        (500, 9, (4, 2, 2)), (512, 16, (64, 9, 2)), (512, 8, (32, 4, 2)), (1000, 8, (8, 4, 2))])
def test_route_scored_many_rows(E, k, groups):
    """From 8192 rows on a row has 16 lanes: 96 rows (ties, absent experts and padding among them), each
    86 times over, in another order of rows for each."""
    logits = normal(96, E, E + k)
    rng = np.random.default_rng(E)
    logits[3] = 0.0
    logits[4] = np.round(logits[4] * 4) / 4
    logits[5, rng.permutation(E)[3:]] = -np.inf
    logits[6] = -np.inf
    logits[7] = torch.from_numpy(logits[7]).to(torch.bfloat16).float().numpy()
    logits[8] = logits[8, 0] + np.arange(E, dtype=np.float32) * np.float32(2.0 ** -22)
    valid = rng.random(96) > 0.1
    logits[~valid] = np.nan
    order = np.concatenate([rng.permutation(96) for _ in range(86)])
    bias = (0.05 * rng.standard_normal(E)).astype(np.float32)
    for scoring, b, renormalise in itertools.product(("softmax", "sigmoid"), (None, bias), (False, True)):
        ids, w = oracle.route_scored(logits, k, scoring, b, *groups, renormalise, 1.5, valid)
        rb = moe.alloc_route_buffers(len(order), E, k, 32)
        moe.route_scored(dev(logits[order]), rb, scoring, dev(b), *groups, renormalise=renormalise, scale=1.5,
                         row_valid=dev(valid[order]))
        np.testing.assert_array_equal(rb.topk_ids.cpu().numpy(), ids[order])
        n = weight_roundings(logits, scoring, renormalise)
        np.testing.assert_allclose(rb.topk_weights.cpu().numpy(), w[order], rtol=n * U, atol=2.0 ** -126)
    check_grouping(rb, ids[order], E)


@pytest.mark.parametrize("scoring", ("softmax", "sigmoid"))
@pytest.mark.parametrize("groups", ((1, 1, 1), (8, 3, 2)))
def test_route_scored_ties_and_neighbours(scoring, groups):
    """Values closer than fp32 scores can tell: equal logits, neighbouring fp32
    numbers, and biases that nearly make up for a difference of scores."""
    rng = np.random.default_rng(5)
    M, E, k = 96, 64, 6
    logits = np.zeros((M, E), np.float32)
    for t in range(M):
        kind = t % 6
        if kind == 0:
            logits[t] = rng.integers(0, 3, E)  # many equal ones
        elif kind == 1:
            logits[t] = np.float32(1.5)  # all equal
        elif kind == 2:
            v = np.full(E, 2.0, np.float32)
            for _ in range(3):
                v = np.where(rng.random(E) < 0.5, np.nextafter(v, np.float32(9)), v)
            logits[t] = v
        elif kind == 3:
            logits[t] = normal(1, E, t)[0]
            logits[t, 40:] = logits[t, :24]
        elif kind == 4:
            logits[t] = -np.abs(normal(1, E, t)[0]) * 1e-7
        else:
            logits[t] = torch.from_numpy(normal(1, E, t)).to(torch.bfloat16).float().numpy()[0]
    check(logits, k, scoring, None, groups)
    check(logits, k, scoring, np.zeros(E, np.float32), groups)
    check(logits, k, scoring, (rng.integers(0, 2, E) * 2.0 ** -20).astype(np.float32), groups)
    # c equal to within some 1e-9: the bias is the rounded difference of two scores
    lg = np.tile(normal(1, E, 77), (M, 1))
    s = oracle.scores(lg[0].astype(np.float64), scoring)
    bias = (s.max() - s).astype(np.float32)
    check(lg, k, scoring, bias, groups)
    lg2 = lg + rng.integers(-2, 3, lg.shape).astype(np.float32) * np.float32(2.0 ** -22)
    check(lg2.astype(np.float32), k, scoring, bias, groups)


@pytest.mark.parametrize("scoring,biased,groups", [("softmax", False, (1, 1, 1)), ("sigmoid", True, (1, 1, 1)),
                                                   ("sigmoid", False, (6, 2, 2)), ("softmax", True, (6, 2, 1)),
                                                   ("softmax", False, (6, 2, 1))])
def test_route_scored_masked_experts(scoring, biased, groups):
    """-inf in logits and biases: absent experts, rows with fewer than k left,
    rows and groups with none, the type's lowest value, infinities and NaN."""
    rng = np.random.default_rng(6)
    M, E, k = 70, 96, 5
    logits = normal(M, E, 6)
    for t in range(M):
        left = [E, 90, 6, 5, 4, 1, 0][t % 7]
        logits[t, rng.permutation(E)[left:]] = -np.inf
    logits[7, 3:9] = np.finfo(np.float32).min
    logits[8] = np.where(np.isinf(logits[8]), np.finfo(np.float32).min, logits[8])
    logits[14, 50] = np.nan
    bias = None
    if biased:
        bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
        bias[10:14] = -np.inf
        bias[40] = -0.5
    with np.errstate(invalid="ignore"):
        for renormalise in (True, False):
            check(logits, k, scoring, bias, groups, renormalise)
            if groups[0] == 1 and not biased:
                x = normal(4, E, 9)
                x[1, 17], x[2, 95], x[2, 4] = np.nan, np.nan, np.nan
                check(x, k, scoring, bias, groups, renormalise)


@pytest.mark.parametrize("groups", ((1, 1, 1), (8, 3, 1), (8, 3, 2)))
def test_route_scored_large_biases_close_together(groups):
    """A few biases far above the others (100, whose fp32 sums are 4e-6 off) and nearly equal c among
    them; of both signs within a group, so that a group's sum is smaller than its terms' errors."""
    rng = np.random.default_rng(70)
    M, E, k = 400, 64, 6
    logits = normal(M, E, 71)
    bias = (0.05 * rng.standard_normal(E)).astype(np.float32)
    s = 1 / (1 + np.exp(-logits[0].astype(np.float64)))
    logits[:200] = logits[0] + rng.integers(-3, 4, (200, E)).astype(np.float32) * np.float32(2.0 ** -18)
    for where, value in ((rng.permutation(E)[:5], 100.0), (np.arange(0, E, 8), 100.0), (np.arange(1, E, 8), -100.0)):
        bias[where] = (value - s[where]).astype(np.float32)
        check(logits, k, "sigmoid", bias, groups, False)
    rest = np.setdiff1d(np.arange(E), np.concatenate([np.arange(0, E, 8), np.arange(1, E, 8)]))
    bias[rest] = -100.0 - 0.01 * rng.random(len(rest)).astype(np.float32)
    check(logits, k, "sigmoid", bias, groups, False)
    bias[rest] = -np.inf  # the two left in a group add up to nearly 0
    check(logits, k, "sigmoid", bias, groups, False)
    bias[rest] = -1e6
    check(logits, k, "sigmoid", bias, groups, False)


def test_route_scored_groups_of_saturated_scores():
    """Logits whose scores are the same in fp64: without a bias the logits decide, between groups as well."""
    M, E, k = 40, 48, 5
    rng = np.random.default_rng(72)
    for logits in (50 + 9 * rng.random((M, E)), -800 - 9 * rng.random((M, E)), 1e-20 * rng.standard_normal((M, E))):
        lg = logits.astype(np.float32)
        for bad in (False, True):
            if bad:
                lg[:, 7] = -np.inf  # (by the exact path)
            for scoring in ("sigmoid", "softmax"):
                check(lg, k, scoring, None, (6, 2, 1))
                if scoring == "softmax" or lg.max() > -700:
                    check(lg, k, scoring, None, (6, 2, 2), False)


def test_route_scored_nan_bias_and_infinite_logits():
    """A NaN bias or logit counts as the highest c; +inf saturates a sigmoid and makes a softmax NaN."""
    M, E, k = 12, 80, 4
    logits = normal(M, E, 60)
    bias = (0.1 * normal(1, E, 61))[0]
    bias[[70, 3]] = np.nan
    logits[3, 50], logits[4, [9, 11]] = np.inf, np.inf
    logits[5, 20] = -np.inf
    with np.errstate(invalid="ignore", over="ignore"):
        for groups in ((1, 1, 1), (8, 2, 2)):
            want, w = oracle.route_scored(logits, k, "sigmoid", bias, *groups, True)
            rb = moe.alloc_route_buffers(M, E, k, 16)
            moe.route_scored(dev(logits), rb, "sigmoid", dev(bias), *groups)
            np.testing.assert_array_equal(rb.topk_ids.cpu().numpy(), want)
            np.testing.assert_allclose(rb.topk_weights.cpu().numpy(), w, rtol=14 * U)
        check(logits, k, "sigmoid", None, (8, 2, 2))
        rb = moe.route_scored(dev(logits), moe.alloc_route_buffers(M, E, k, 16), renormalise=False)
        got = rb.topk_weights.cpu().numpy()
        assert np.isnan(got[[3, 4]]).all() and np.isfinite(got[[0, 1, 2, 5]]).all()
        assert rb.topk_ids[3, 0] == 50 and rb.topk_ids[4, :2].tolist() == [9, 11]


def test_route_scored_more_rows_than_a_grid():
    """More rows than one launch's workgroups take (2^23 of 16 rows)."""
    M, E = 2**27 + 21, 2
    logits = torch.zeros((M, E), device="cuda")
    logits[::3, 1] = 1.0
    rb = moe.alloc_route_buffers(M, E, 1, 16)
    moe.route_scored(logits, rb, "sigmoid", renormalise=False, grouping=False)
    want = torch.zeros(M, dtype=torch.int32, device="cuda")
    want[::3] = 1
    assert torch.equal(rb.topk_ids[:, 0], want)
    assert (rb.topk_weights[:, 0] - torch.where(want == 1, 1 / (1 + np.exp(-1.0)), 0.5)).abs().max() <= 4 * U
    grad = moe.route_scored_backward(logits, rb.topk_ids, torch.ones((M, 1), device="cuda"), "sigmoid", False)
    other = grad.gather(1, 1 - want[:, None].long())
    assert not other.any() and (grad[:, 0][1::3] - 0.25).abs().max() <= 4 * U


def test_route_scored_large_values():
    """Logits and biases of every magnitude: the scores saturate, and fp32 errors
    of c grow with the bias."""
    rng = np.random.default_rng(8)
    E, k = 48, 4
    rows = [normal(1, E, 10 + i)[0] * np.float32(10.0 ** i) for i in range(0, 30, 3)]
    rows += [normal(1, E, 50)[0] + np.float32(v) for v in (50.0, -50.0, 3e6, -3e6, 1e30, -1e30)]
    logits = np.stack(rows).astype(np.float32)
    for scoring in ("softmax", "sigmoid"):
        for bias in (None, (1e3 * rng.standard_normal(E)).astype(np.float32),
                     np.where(rng.random(E) < 0.5, np.float32(1e6), np.float32(1e6 + 0.0625)).astype(np.float32)):
            M = logits.shape[0]
            want, w = oracle.route_scored(logits, k, scoring, bias, renormalise=False)
            rb = moe.alloc_route_buffers(M, E, k, 16)
            moe.route_scored(dev(logits), rb, scoring=scoring, bias=dev(bias), renormalise=False)
            np.testing.assert_array_equal(rb.topk_ids.cpu().numpy(), want)
            for t in range(M):
                # probabilities below 2^-126 apart, differences up to 104 are rounded
                n = (2 * min(spread_of(logits[t]), 104.0) + 20) if scoring == "softmax" else 10
                np.testing.assert_allclose(rb.topk_weights[t].cpu().numpy(), w[t], rtol=n * U, atol=2.0 ** -120)


def test_route_scored_one_launch_and_two_agree():
    """16 rows are grouped in the routing's launch, 17 by the grouping kernel, 4096
    assignments by a grid; a workgroup's rows do not depend on the others'."""
    E, k = 256, 8
    logits = normal(600, E, 11)
    bias = (0.05 * np.random.default_rng(1).standard_normal(E)).astype(np.float32)
    big = check(logits, k, "sigmoid", bias, (8, 4, 2), block=32)
    for M in (1, 15, 16, 17, 33):
        rb = check(logits[:M], k, "sigmoid", bias, (8, 4, 2), block=32)
        assert torch.equal(rb.topk_ids, big.topk_ids[:M]) and torch.equal(rb.topk_weights, big.topk_weights[:M])


def test_route_scored_buffers_of_a_larger_batch():
    """cap above what the batch can reach: all of it is written, and nothing past it."""
    M, E, k, block = 20, 32, 3, 16
    logits = normal(M, E, 12)
    big = moe.alloc_route_buffers(200, E, k, block)
    for rows in (M, 9):
        room = torch.full((big.cap + 8,), 5, dtype=torch.int32, device="cuda")
        blocks = torch.full((big.cap // block + 8,), 5, dtype=torch.int32, device="cuda")
        ids = torch.full((rows, k), 5, dtype=torch.int32, device="cuda")
        w = torch.zeros((rows, k), device="cuda")
        moe.moe_route_scored(dev(logits[:rows]), k, ids, w, block_m=block, sorted_token_ids=room, block_expert_ids=blocks,
                             expert_offsets=big.expert_offsets, num_tokens_post_pad=big.num_tokens_post_pad, cap=big.cap)
        npp = int(big.num_tokens_post_pad.item())
        assert (room[npp:big.cap] == rows * k).all() and (room[big.cap:] == 5).all()
        nb = npp // block
        assert (blocks[:nb] >= 0).all() and (blocks[nb:big.cap // block] == -1).all() and (blocks[big.cap // block:] == 5).all()


def test_route_scored_unaligned():
    M, E, k = 21, 64, 4
    logits = normal(M, E, 13)
    room = torch.zeros(M * E + 1, device="cuda")
    view = room[1:].view(M, E)
    view.copy_(dev(logits))
    b = torch.zeros(E + 1, device="cuda")[1:]
    b.copy_(dev((0.1 * normal(1, E, 3))[0]))
    rb, want = moe.alloc_route_buffers(M, E, k, 16), moe.alloc_route_buffers(M, E, k, 16)
    moe.route_scored(view, rb, scoring="sigmoid", bias=b, n_groups=4, top_groups=2)
    moe.route_scored(dev(logits), want, scoring="sigmoid", bias=b.clone(), n_groups=4, top_groups=2)
    assert torch.equal(rb.topk_ids, want.topk_ids) and torch.equal(rb.topk_weights, want.topk_weights)


@pytest.mark.parametrize("M,drop", [(1, 0.0), (1, 1.0), (12, 0.4), (70, 0.5), (70, 1.0), (600, 0.3), (600, 1.0)])
def test_dropped_rows_through_the_layer(M, drop):
    """Padding rows and absent experts cost the experts no rows and give zeros."""
    s = wl.LayerShape(E=16, H=512, I=256, k=3)
    layer = device_layer(s, 3)
    t = wl.tokens(s, M, 30 + M)
    valid = np.random.default_rng(M).random(M) >= drop
    logits = t.logits.copy()
    logits[::3, 5:] = -np.inf
    logits[1::7, 1:] = -np.inf  # one expert left
    block = moe.moe_w4a16_preferred_block_m(M, s.E, s.H, s.I, s.k)
    rb = check(logits, s.k, "sigmoid", None, (1, 1, 1), True, 2.0, valid, block)
    out = moe.forward(x_device(t.x_bits), rb, s.I, layer.w13, layer.w2).float().cpu().numpy()
    ids, w = rb.topk_ids.cpu().numpy(), rb.topk_weights.cpu().numpy().astype(np.float64)
    x = wl.f32_from_bf16_bits(t.x_bits).astype(np.float64)
    cache = oracle_experts(s, 3)
    want = np.zeros((M, s.H))
    for row in range(M):
        left = ids[row] >= 0
        if left.any():
            want[row] = oracle.moe_forward(x[row:row + 1], ids[row:row + 1, left], w[row:row + 1, left], cache)[0]
    assert not out[~valid].any()
    if drop < 1.0:
        assert_output_close(out, want)


def test_balance_loss_leaves_dropped_slots_out():
    M, E, k = 50, 24, 4
    logits = normal(M, E, 14)
    valid = np.random.default_rng(2).random(M) > 0.3
    rb = moe.alloc_route_buffers(M, E, k, 16)
    moe.route_scored(dev(logits), rb, row_valid=dev(valid))
    bufs = moe.balance_loss(dev(logits), rb.topk_ids, moe.alloc_balance_buffers(M, E), row_valid=dev(valid))
    want = oracle.balance(logits, rb.topk_ids.cpu().numpy(), None, valid)
    np.testing.assert_array_equal(bufs.expert_counts.cpu().numpy(), want["counts"])


def check_backward(logits, ids, scoring, renormalise, scale=1.0, base=None, seed=3, in_place=False):
    M, E = logits.shape
    g = np.random.default_rng(seed).standard_normal(ids.shape).astype(np.float32)
    want, mag = oracle.route_scored_backward(logits, ids, g, scoring, renormalise, scale, base)
    b = dev(base)
    out = b if in_place else torch.full((M, E), -5.0, device="cuda")
    got = moe.route_scored_backward(dev(logits), dev(ids), dev(g), scoring=scoring, renormalise=renormalise, scale=scale,
                                    grad_base=b, grad_logits=out).cpu().numpy()
    # twice a weight's roundings (the slot's own and those in the sum), the products, the difference, the sum's 4
    n = 2 * weight_roundings(logits, scoring, renormalise) + 12
    bound = n * U * mag + U * (0 if base is None else np.abs(want)) + 2.0 ** -120
    assert (np.abs(got - want) <= bound).all(), np.max(np.abs(got - want) / bound)
    return got


@pytest.mark.parametrize("M,E,k", [(1, 1, 1), (1, 384, 8), (33, 60, 4), (17, 9, 9), (200, 128, 8), (65, 257, 5),
                                   (40, 500, 16), (31, 1024, 16), (9, 1021, 3)])
def test_route_scored_backward_shapes(M, E, k):
    logits = normal(M, E, 20 + M)
    rng = np.random.default_rng(M)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(M)]).astype(np.int32)
    for i, (scoring, renormalise) in enumerate(itertools.product(("softmax", "sigmoid"), (False, True))):
        base = rng.standard_normal((M, E)).astype(np.float32) if i % 2 else None
        some = ids.copy()
        some[rng.random(ids.shape) < 0.2] = rng.choice([-1, E, 2**31 - 1, -2**31])
        check_backward(logits, ids, scoring, renormalise, 2.5, base)
        check_backward(logits, some, scoring, renormalise, 2.5, base)
        check_backward(logits, some, scoring, renormalise, 1.0, rng.standard_normal((M, E)).astype(np.float32), in_place=True)


def test_route_scored_backward_rows_without_experts():
    """Padding rows hold NaN; they have no gradient, and the base passes through."""
    M, E, k = 20, 40, 3
    logits = normal(M, E, 30)
    ids = np.tile(np.arange(k, dtype=np.int32), (M, 1))
    ids[5:9] = -1
    logits[5:9] = np.nan
    base = np.random.default_rng(1).standard_normal((M, E)).astype(np.float32)
    for scoring, renormalise in itertools.product(("softmax", "sigmoid"), (False, True)):
        for in_place in (False, True):
            got = check_backward(logits, ids, scoring, renormalise, base=base, in_place=in_place)
            np.testing.assert_array_equal(got[5:9], base[5:9])
    # absent experts keep a zero gradient
    logits = normal(M, E, 31)
    logits[:, 20:] = -np.inf
    got = check_backward(logits, ids, "softmax", False)
    assert not got[:, 20:].any()


def test_route_scored_backward_far_logits():
    logits = normal(6, 32, 32) * np.float32(1.0)
    logits[1] += 80
    logits[2] -= 80
    logits[3] *= 30
    logits[4, 3] = 200
    logits[5] = -200  # sigmoid scores below the smallest fp32 number: no gradient
    ids = np.tile(np.array([3, 9, 1], np.int32), (6, 1))
    for scoring, renormalise in itertools.product(("softmax", "sigmoid"), (False, True)):
        check_backward(logits, ids, scoring, renormalise)


@pytest.mark.parametrize("M,E,groups", [(5, 48, (1, 1, 1)), (40, 48, (6, 2, 2)), (60, 384, (1, 1, 1))])
def test_route_scored_sigmoids_below_the_normal_numbers(M, E, groups):
    """Scores that fp32 holds as subnormal numbers or not at all: weights and gradients made of them have all
    their bits (renormalised, they are divided by 1e-20)."""
    base = normal(M, E, 80)
    rng = np.random.default_rng(81)
    ids = np.stack([rng.permutation(E)[:4] for _ in range(M)]).astype(np.int32)
    for shift in (-80.0, -86.0, -92.0, -100.0, -120.0):
        logits = base + np.float32(shift)
        mixed = logits.copy()
        mixed[:, ::3] = base[:, ::3] - 40  # beside others
        for lg in (logits, mixed):
            for renormalise, scale in ((True, 2.5), (False, 1.0), (False, 1e9)):
                want_ids, want = oracle.route_scored(lg, 4, "sigmoid", None, *groups, renormalise, scale)
                rb = moe.route_scored(dev(lg), moe.alloc_route_buffers(M, E, 4, 16), "sigmoid", None, *groups,
                                      renormalise=renormalise, scale=scale)
                np.testing.assert_array_equal(rb.topk_ids.cpu().numpy(), want_ids)
                # the exponential of half the logit counts twice, and a product more joins the halves
                n = weight_roundings(lg, "sigmoid", renormalise) + 3
                np.testing.assert_allclose(rb.topk_weights.cpu().numpy(), want, rtol=n * U, atol=2.0 ** -126)
                check_backward(lg, ids, "sigmoid", renormalise, scale)
                check_backward(-lg, ids, "sigmoid", renormalise, scale)  # the slope is as small


def test_route_scored_backward_is_the_forwards_difference():
    """The gradient against differences of the device's own fp32 forward (E = 6,
    step 2^-7: its third derivatives are below 1, so off by at most 2^-14 / 6
    of them and 2 roundings of 10 x 2^-24 over the step)."""
    M, E, k, h = 4, 6, 2, 2.0 ** -7
    logits = np.round(normal(M, E, 33) * 64) / 64
    for scoring, renormalise in itertools.product(("softmax", "sigmoid"), (False, True)):
        def weights(lg, ids):
            rb = moe.alloc_route_buffers(M, E, k, 16)
            moe.route_scored(dev(lg.astype(np.float32)), rb, scoring=scoring, renormalise=renormalise)
            at = rb.topk_ids.cpu().numpy()
            if ids is None:
                return at
            w = rb.topk_weights.cpu().numpy().astype(np.float64)
            return np.array([[w[t][list(at[t]).index(e)] if e in at[t] else np.nan for e in ids[t]] for t in range(M)])
        ids = weights(logits, None)
        g = np.random.default_rng(4).standard_normal((M, k)).astype(np.float32)
        got = moe.route_scored_backward(dev(logits.astype(np.float32)), dev(ids.astype(np.int32)), dev(g), scoring=scoring,
                                        renormalise=renormalise).cpu().numpy()
        for e in range(E):
            up, down = logits.copy(), logits.copy()
            up[:, e] += h
            down[:, e] -= h
            d = ((weights(up, ids) - weights(down, ids)) * g).sum(1) / (2 * h)
            ok = ~np.isnan(d)  # (the step changed the choice)
            assert ok.sum() >= M - 2
            tol = (h * h / 6 + 2 * 10 * U / (2 * h)) * np.abs(g).sum(1)
            assert (np.abs(got[:, e] - d)[ok] <= tol[ok]).all()


def test_route_scored_same_bits_streams_and_replays():
    M, E, k = 700, 160, 6
    logits = normal(M, E, 40)
    lg, b = dev(logits), dev((0.05 * normal(1, E, 2))[0])
    valid = dev(np.random.default_rng(3).random(M) > 0.1)
    rb, small = moe.alloc_route_buffers(M, E, k, 32), moe.alloc_route_buffers(16, E, k, 16)
    gw, grad = torch.randn((M, k), device="cuda"), torch.zeros((M, E), device="cuda")
    base = torch.randn((M, E), device="cuda")

    def call(stream=None):
        moe.route_scored(lg, rb, "sigmoid", b, 8, 3, 2, row_valid=valid, stream=stream)
        moe.route_scored(lg[:16], small, "softmax", b, stream=stream)
        moe.route_scored_backward(lg, rb.topk_ids, gw, "sigmoid", grad_base=base, grad_logits=grad, stream=stream)
        return [rb.topk_ids, rb.topk_weights, rb.sorted_token_ids, rb.block_expert_ids, rb.expert_offsets,
                rb.num_tokens_post_pad, small.topk_ids, small.topk_weights, small.sorted_token_ids, grad]

    first = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, call()))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = call()
    for rep in range(4):
        lg.copy_(dev(logits) * (1 + rep % 2))
        for t in outs:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in outs]
        assert all(torch.equal(x, y) for x, y in zip(replayed, call()))
        if rep % 2 == 0:
            assert all(torch.equal(x, y) for x, y in zip(replayed, first))


def test_route_scored_offsets_past_32_bits():
    """M * E > 2^32 values: the last rows' choices and gradients."""
    E, k = 1024, 4
    M = 2**22 + 40
    logits = torch.zeros((M, E), device="cuda")
    tail = normal(48, E, 50)
    logits[-48:] = dev(tail)
    rb = moe.alloc_route_buffers(M, E, k, 16)
    moe.route_scored(logits, rb, "sigmoid", renormalise=False, grouping=False)
    want, w = oracle.route_scored(tail, k, "sigmoid", renormalise=False)
    np.testing.assert_array_equal(rb.topk_ids[-48:].cpu().numpy(), want)
    np.testing.assert_allclose(rb.topk_weights[-48:].cpu().numpy(), w, rtol=10 * U)
    assert rb.topk_ids[:M - 48].eq(torch.arange(k, device="cuda", dtype=torch.int32)).all()
    gw = torch.ones((M, k), device="cuda")
    grad = moe.route_scored_backward(logits, rb.topk_ids, gw, "softmax", False)
    full, _ = oracle.route_scored_backward(tail, want, np.ones((48, k)), "softmax", False)
    np.testing.assert_allclose(grad[-48:].cpu().numpy(), full, atol=1e-6)  # (against a wrong row, not roundings)


def test_route_scored_wrapper_refusals():
    lg = torch.zeros((4, 8), device="cuda")
    rb = moe.alloc_route_buffers(4, 8, 2, 16)
    gw = torch.zeros((4, 2), device="cuda")
    for bad in (lambda: moe.route_scored(lg.double(), rb), lambda: moe.route_scored(lg[:3], rb),
                lambda: moe.route_scored(lg, rb, scoring="tanh"), lambda: moe.route_scored(lg.t(), rb),
                lambda: moe.route_scored(lg, rb, bias=torch.zeros(7, device="cuda")),
                lambda: moe.route_scored(lg, rb, bias=torch.zeros(8)),
                lambda: moe.route_scored(lg.cpu(), rb),
                lambda: moe.route_scored(lg, rb, row_valid=torch.ones(3, dtype=torch.bool, device="cuda")),
                lambda: moe.route_scored_backward(lg, rb.topk_ids, gw[:3]),
                lambda: moe.route_scored_backward(lg, rb.topk_ids.long(), gw),
                lambda: moe.route_scored_backward(lg, rb.topk_ids, gw, grad_base=lg.t().contiguous().t())):
        with pytest.raises(ValueError):
            bad()
    for bad in (dict(n_groups=3), dict(n_groups=8, top_groups=1), dict(n_groups=4, top_groups=2, group_top=3)):
        with pytest.raises(moe.MoeError):
            moe.route_scored(lg, rb, **bad)
