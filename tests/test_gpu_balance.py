"""Balance loss, counts and gradient against the float64 oracle.

Tolerances count roundings of 2^-24 (fp32, half a step). A probability
exp(l - m) / s carries |l - m| of them from the rounded difference, 4 from
the exponential and 2 from the division, and the row's sum one for each of
the values a lane adds (E / 16, rounded up to 64s) and 4 to join the lanes.
A chunk's sum of probabilities adds one for each row of a lane (at most
M / 8192 + 1: chunks of M / 256 rows, of which a pass takes 32 or 64), 2 to join
a wave's rows and 15 its 16 waves; the final sum is fp64."""
import numpy as np
import pytest
import torch

import int4_weight_only_moe_amd as moe
import oracle

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def row_roundings(logits, E):
    live = logits[np.isfinite(logits)]
    spread = float(live.max() - live.min()) if live.size else 0.0
    return spread + 6 + 4 * (-(-E // 64)) + 4


def make(M, E, k, S, masked, seed):
    rng = np.random.default_rng(seed)
    logits = (rng.standard_normal((M, E)) + rng.standard_normal(E)).astype(np.float32)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(M)]).astype(np.int32) if M else np.zeros((0, k), np.int32)
    off = np.sort(rng.integers(0, M + 1, S + 1)).astype(np.int32) if S > 1 else None
    valid = rng.random(M) > 0.25 if masked else None
    if masked and M:
        logits[~valid] = np.nan
        ids[~valid] = rng.integers(-2**31, 2**31, ids[~valid].shape)
    return logits, ids, off, valid


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def check(logits, ids, off, valid, E, k, S):
    M = logits.shape[0]
    ref = oracle.balance(logits, ids, off, valid)
    bufs = moe.alloc_balance_buffers(M, E, S)
    for t in (bufs.expert_counts, bufs.seq_tokens, bufs.workspace):
        t.fill_(77)
    bufs.prob_sums.fill_(7.0)
    bufs.loss.fill_(7.0)
    moe.balance_loss(dev(logits), dev(ids), bufs, seq_offsets=dev(off), row_valid=dev(valid))
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bufs.expert_counts.cpu().numpy(), ref["counts"])
    np.testing.assert_array_equal(bufs.seq_tokens.cpu().numpy(), ref["tokens"])
    rtol = (row_roundings(logits, E) + M / 8192 + 1 + 2 + 15 + 1) * U
    np.testing.assert_allclose(bufs.prob_sums.cpu().numpy(), ref["probs"], rtol=rtol, atol=2.0 ** -126)
    np.testing.assert_allclose(bufs.loss.cpu().numpy(), ref["loss"], rtol=rtol + U, atol=2.0 ** -126)
    return bufs, ref


def check_backward(logits, off, valid, E, k, S, counts, tokens, seed=3):
    M = logits.shape[0]
    rng = np.random.default_rng(seed)
    gl = rng.standard_normal(S).astype(np.float32)
    want = oracle.balance_backward(logits, k, counts, tokens, gl, off, valid)
    got = torch.full((M, E), -5.0, device="cuda")
    moe.balance_loss_backward(dev(logits), k, dev(counts.astype(np.int32)), dev(tokens.astype(np.int32)), dev(gl),
                              seq_offsets=dev(off), row_valid=dev(valid), grad_logits=got)
    got = got.cpu().numpy()
    outside = np.isnan(want)
    assert (got[outside] == -5.0).all()
    # |w| p (c + sum c p) bounds what the rounded terms can be off: p's own
    # roundings twice, the dot's adds, the difference, three products
    bound = np.zeros((M, E))
    offs = [0, M] if off is None else list(off)
    for s in range(S):
        for t in range(offs[s], offs[s + 1]):
            if valid is None or valid[t]:
                p = oracle._softmax_or_zero(logits[t].astype(np.float64))
                bound[t] = abs(gl[s]) * E / (k * float(tokens[s]) ** 2) * p * (counts[s] + counts[s] @ p)
    n = 2 * row_roundings(logits, E) + 4 * (-(-E // 64)) + 4 + 10
    err = np.abs(np.where(outside, 0, got - np.where(outside, 0, want)))
    assert (err[~outside] <= (n * U * bound + 2.0 ** -126)[~outside]).all(), float((err / (bound * U + 1e-300))[~outside].max())
    return got


CASES = [
    # M, E, k, S, masked
    (1, 1, 1, 1, False), (1, 8, 2, 1, True), (3, 8, 8, 1, False), (17, 60, 4, 1, False), (40, 64, 8, 5, True),
    (64, 65, 3, 1, True), (100, 128, 8, 3, False), (130, 130, 6, 40, True), (257, 256, 8, 2, True),
    (300, 384, 8, 1, False), (1000, 384, 8, 7, True), (90, 500, 16, 2, False), (120, 512, 8, 33, True),
    (77, 700, 8, 1, True), (200, 1024, 8, 2, False), (129, 1021, 16, 3, True), (9000, 8, 2, 4, True),
    (20000, 16, 2, 1, False),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_balance_matches_oracle(case):
    M, E, k, S, masked = CASES[case]
    logits, ids, off, valid = make(M, E, k, S, masked, 100 + case)
    _, ref = check(logits, ids, off, valid, E, k, S)
    check_backward(logits, off, valid, E, k, S, ref["counts"], ref["tokens"])


def test_balance_of_no_rows_is_zero():
    check(*make(0, 12, 3, 1, False, 0), 12, 3, 1)
    bufs = moe.alloc_balance_buffers(0, 12, 1)
    out = torch.empty((0, 12), device="cuda")
    assert moe.balance_loss_backward(out, 3, bufs.expert_counts, bufs.seq_tokens, bufs.loss).shape == (0, 12)


def test_balance_all_rows_masked_and_empty_sequences():
    logits, ids, _, _ = make(30, 20, 2, 1, False, 1)
    off = np.array([0, 0, 10, 10, 30, 30], np.int32)
    valid = np.arange(30) < 10
    logits[~valid] = np.nan
    bufs, ref = check(logits, ids, off, valid, 20, 2, 5)
    assert bufs.seq_tokens.tolist() == [0, 10, 0, 0, 0]
    got = check_backward(logits, off, valid, 20, 2, 5, ref["counts"], ref["tokens"])
    assert (got[10:] == 0).all()


def test_balance_infinite_and_dropped():
    """-inf logits (masked experts), rows of nothing else, choices that were dropped, the type's lowest value."""
    logits, ids, _, _ = make(50, 70, 4, 1, False, 2)
    logits[:, 5:9] = -np.inf
    logits[7] = -np.inf
    logits[8] = np.finfo(np.float32).min  # a row of the lowest value: uniform
    logits[9, 1:] = -np.inf  # one expert left
    logits[10, :35] = -np.inf
    ids[3] = -1
    ids[4, 2] = 70
    ids[5, 1] = np.iinfo(np.int32).min
    rows = [r for r in range(50) if r != 8]  # the lowest value would enter the tolerance's spread
    bufs, ref = check(logits[rows], ids[rows], None, None, 70, 4, 1)
    got = check_backward(logits[rows], None, None, 70, 4, 1, ref["counts"], ref["tokens"])
    assert (got[7] == 0).all() and (got[:, 5:9] == 0).all()
    one = moe.alloc_balance_buffers(1, 70)
    moe.balance_loss(dev(logits[8:9]), dev(ids[8:9]), one)
    np.testing.assert_allclose(one.prob_sums.cpu().numpy(), 1 / 70, rtol=80 * U)


def test_balance_nan_in_a_valid_row_shows():
    logits, ids, _, _ = make(40, 64, 4, 1, False, 4)
    logits[11, 3] = np.nan
    logits[11, 4:] = -np.inf
    bufs = moe.alloc_balance_buffers(40, 64)
    moe.balance_loss(dev(logits), dev(ids), bufs)
    assert torch.isnan(bufs.loss).all()


def test_balance_unaligned_logits():
    """A view that starts 4 bytes off a 16-byte boundary takes the scalar loads."""
    M, E, k = 33, 64, 4
    logits, ids, _, _ = make(M, E, k, 1, False, 8)
    room = torch.zeros(M * E + 1, device="cuda")
    view = room[1:].view(M, E)
    view.copy_(dev(logits))
    assert view.data_ptr() % 16 == 4
    a, b = moe.alloc_balance_buffers(M, E), moe.alloc_balance_buffers(M, E)
    moe.balance_loss(view, dev(ids), a)
    moe.balance_loss(dev(logits), dev(ids), b)
    assert torch.equal(a.prob_sums, b.prob_sums) and torch.equal(a.loss, b.loss)
    gl = torch.ones(1, device="cuda")
    out = torch.zeros(M * E + 1, device="cuda")
    g = moe.balance_loss_backward(view, k, a.expert_counts, a.seq_tokens, gl, grad_logits=out[1:].view(M, E))
    assert torch.equal(g, moe.balance_loss_backward(dev(logits), k, a.expert_counts, a.seq_tokens, gl))
    assert out[0] == 0


def test_balance_same_bits_on_every_call_streams_and_replays():
    M, E, k, S = 3000, 160, 6, 3
    logits, ids, off, valid = make(M, E, k, S, True, 9)
    lg, iv, ov, va = dev(logits), dev(ids), dev(off), dev(valid)
    bufs = moe.alloc_balance_buffers(M, E, S)
    gl = torch.randn(S, device="cuda")
    grad = torch.zeros_like(lg)

    def call(stream=None):
        moe.balance_loss(lg, iv, bufs, seq_offsets=ov, row_valid=va, stream=stream)
        moe.balance_loss_backward(lg, k, bufs.expert_counts, bufs.seq_tokens, gl, seq_offsets=ov, row_valid=va,
                                  grad_logits=grad, stream=stream)
        return bufs.loss, bufs.prob_sums, grad

    first = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (bufs.loss, bufs.prob_sums, grad)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for rep in range(4):
        lg.copy_(dev(logits) * (1 + rep % 2))
        for t in (bufs.loss, bufs.prob_sums, bufs.workspace, grad):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in (bufs.loss, bufs.prob_sums, grad)]
        assert all(torch.equal(a, b) for a, b in zip(replayed, call()))
        if rep % 2 == 0:
            assert all(torch.equal(a, b) for a, b in zip(replayed, first))


def test_balance_wrapper_refusals():
    lg = torch.zeros((4, 8), device="cuda")
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    bufs = moe.alloc_balance_buffers(4, 8)
    for bad in (lambda: moe.balance_loss(lg.double(), ids, bufs), lambda: moe.balance_loss(lg, ids.long(), bufs),
                lambda: moe.balance_loss(lg.t().contiguous().t(), ids, bufs),
                lambda: moe.balance_loss(lg, ids[:3], bufs), lambda: moe.balance_loss(lg, ids.cpu(), bufs),
                lambda: moe.balance_loss(lg, ids, bufs, row_valid=torch.ones(3, dtype=torch.bool, device="cuda")),
                lambda: moe.balance_loss(lg, ids, bufs, seq_offsets=torch.zeros(3, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    small = moe.alloc_balance_buffers(4, 8)
    small.workspace = small.workspace[:16]
    with pytest.raises(moe.MoeError) as e:
        moe.balance_loss(lg, ids, small)
    assert e.value.status == moe.MOE_ERR_WORKSPACE


def test_balance_many_short_sequences_and_one_workgroup():
    """Up to 128 rows and 64 sequences one workgroup does it all; around that limit the same results."""
    for M, S in ((128, 64), (128, 65), (129, 3), (5, 64), (2000, 1999)):
        rng = np.random.default_rng(M + S)
        logits, ids, _, valid = make(M, 48, 4, 1, True, 200 + M)
        off = np.concatenate([[0], np.sort(rng.integers(0, M + 1, S - 1)), [M]]).astype(np.int32)
        bufs, ref = check(logits, ids, off, valid, 48, 4, S)
        check_backward(logits, off, valid, 48, 4, S, ref["counts"], ref["tokens"])


def test_balance_large_logits():
    """Rows of every magnitude, each of values a few steps of its type apart:
    a row that a mask has moved as a whole keeps its probabilities. Values more
    than 104 below the maximum are below 2^-126; the others differ by at most
    104, which is what the tolerance counts for a difference."""
    E, k = 24, 2
    tops = [3e6, -3e6, 1e9, -1e9, 1e10, -1e10, 1.7e12, -1e15, 1e20, -1e25, 1e29, -1e30, 1.2e30, -1.3e30, 1e31, 3e38,
            np.finfo(np.float32).min]
    rng = np.random.default_rng(12)
    logits = np.zeros((len(tops), E), np.float32)
    for i, top in enumerate(tops):
        steps = rng.integers(0, 3, E)
        v = np.full(E, top, np.float32)
        for _ in range(2):
            v = np.where(steps > 0, np.nextafter(v, np.float32(0)), v)
            steps -= 1
        logits[i] = v
    logits[4, 5:] = 0.25  # 1e10 against ordinary values
    logits[5, 7] = 0.25
    S = len(tops)
    off = np.arange(S + 1, dtype=np.int32)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(S)]).astype(np.int32)
    ref = oracle.balance(logits, ids, off, None)
    n = 104 + 6 + 4 + 4
    for repeat in (1, 20):  # one workgroup, and the chunks' path
        lg, iv, ov = np.repeat(logits, repeat, 0), np.repeat(ids, repeat, 0), off * repeat
        bufs = moe.alloc_balance_buffers(S * repeat, E, S)
        moe.balance_loss(dev(lg), dev(iv), bufs, seq_offsets=dev(ov))
        np.testing.assert_allclose(bufs.prob_sums.cpu().numpy(), ref["probs"] * repeat, rtol=(n + 10) * U,
                                   atol=repeat * 2.0 ** -126)
        np.testing.assert_allclose(bufs.loss.cpu().numpy(), ref["loss"], rtol=(n + 11) * U, atol=2.0 ** -120)
    gl = np.ones(S, np.float32)
    want = oracle.balance_backward(logits, k, ref["counts"], ref["tokens"], gl, off, None)
    got = moe.balance_loss_backward(dev(logits), k, dev(ref["counts"].astype(np.int32)),
                                    dev(ref["tokens"].astype(np.int32)), dev(gl), seq_offsets=dev(off))
    p = ref["probs"]
    bound = E / k * p * (ref["counts"] + (ref["counts"] * p).sum(1, keepdims=True))
    err = np.abs(got.cpu().numpy() - want)
    assert (err <= (2 * n + 4 + 4 + 10) * U * bound + 2.0 ** -120).all()


def test_balance_most_rows():
    """More rows than a grid of one thread for 8 of them could have threads (2^29)."""
    M, E, k = 2**29 + 777, 2, 1
    logits = torch.randn((M, E), device="cuda")
    ids = torch.zeros((M, k), dtype=torch.int32, device="cuda")
    ids[:M // 3] = 1
    bufs = moe.balance_loss(logits, ids, moe.alloc_balance_buffers(M, E))
    assert bufs.seq_tokens.tolist() == [M] and bufs.expert_counts.tolist() == [[M - M // 3, M // 3]]
    gl = torch.full((1,), float(M), device="cuda")
    grad = torch.full_like(logits, 7.0)
    moe.balance_loss_backward(logits, k, bufs.expert_counts, bufs.seq_tokens, gl, grad_logits=grad)
    counts = bufs.expert_counts.cpu().numpy()
    for lo in (0, M // 2, M - 1000):
        row = logits[lo:lo + 1000].double().cpu().numpy()
        p = np.exp(row - row.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        w = float(M) * E / (k * float(M) ** 2)
        want = w * p * (counts - (counts * p).sum(1, keepdims=True))
        # c, T and E / (k T) are rounded to fp32 too: four roundings more than the small cases
        n = 2 * row_roundings(row, E) + 4 + 4 + 10 + 4
        bound = w * p * (counts + (counts * p).sum(1, keepdims=True))
        assert (np.abs(grad[lo:lo + 1000].cpu().numpy() - want) <= n * U * bound).all()
    step = 1 << 24
    assert all(bool((grad[i:i + step] != 7.0).all()) for i in range(0, M, step))


def balance_on_device(logits, topk_ids, offsets, valid, S):
    """Counts, sums of probabilities, tokens and loss in float64, some rows at a time (logits finite where valid)."""
    M, E = logits.shape
    k = topk_ids.shape[1]
    counts = torch.zeros(S * E, dtype=torch.int64, device="cuda")
    sums = torch.zeros((S, E), dtype=torch.float64, device="cuda")
    tokens = torch.zeros(S, dtype=torch.int64, device="cuda")
    for s in range(S):
        for lo in range(offsets[s], offsets[s + 1], 1 << 20):
            rows = slice(lo, min(lo + (1 << 20), offsets[s + 1]))
            p = torch.softmax(logits[rows].double(), 1)
            live = torch.ones(p.shape[0], dtype=torch.bool, device="cuda") if valid is None else valid[rows]
            sums[s] += p[live].sum(0)
            tokens[s] += live.sum()
            counts[s * E:(s + 1) * E] += torch.bincount(topk_ids[rows][live].long().reshape(-1), minlength=E)
    counts = counts.view(S, E)
    loss = E / (k * tokens.double() ** 2) * (counts * sums).sum(1)
    return counts, sums, tokens, loss


@pytest.mark.parametrize("M,E,k,cuts,masked,spread", [
    (2**26 + 777, 5, 1, (), False, 0.0),       # equal rows: every addition rounds the same way
    (2**26 + 777, 5, 2, (0.3, 0.3, 0.9), True, 4.0),
    (2**22 + 1, 100, 3, (0.5,), False, 0.0),
    (600_001, 516, 4, (0.1, 0.77), True, 2.0),  # 32 lanes a row
])
def test_balance_sums_of_many_rows(M, E, k, cuts, masked, spread):
    """A lane adds at most 64 rows in fp32, whatever the number of rows: 64
    roundings, 2 to join a wave's rows, 15 its waves, and two to fp32 (a chunk's
    sum, the result); the longer sums are fp64. The rows of spread s differ by at
    most s, and the loss is rounded once more."""
    g = torch.Generator(device="cuda").manual_seed(M + E)
    logits = torch.rand((M, E), device="cuda", generator=g).mul_(spread)
    ids = torch.randint(0, E, (M, k), device="cuda", generator=g, dtype=torch.int32)
    S = len(cuts) + 1
    off = [0, *[int(c * M) for c in cuts], M]
    valid = torch.rand(M, device="cuda", generator=g) > 0.1 if masked else None
    want = balance_on_device(logits, ids, off, valid, S)
    if masked:
        logits[~valid] = float("nan")
    bufs = moe.balance_loss(logits, ids, moe.alloc_balance_buffers(M, E, S),
                            torch.tensor(off, dtype=torch.int32, device="cuda") if S > 1 else None, valid)
    assert torch.equal(bufs.expert_counts.long(), want[0]) and torch.equal(bufs.seq_tokens.long(), want[2])
    n = spread + 6 + 4 * (-(-E // 64)) + 4 + 64 + 2 + 15 + 2
    off_by = ((bufs.prob_sums.double() - want[1]).abs() / want[1].clamp(min=1e-30)).max().item()
    loss_off = ((bufs.loss.double() - want[3]).abs() / want[3].clamp(min=1e-30)).nan_to_num(0.0).max().item()
    print(f"sums off by {off_by / U:.1f} roundings, loss by {loss_off / U:.1f}, of {n:.0f}")
    assert off_by <= n * U and loss_off <= (n + 1) * U
