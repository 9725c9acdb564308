"""The global gradient norm and clipping against float64.

sumsq: the squares and sums are fp64; a thread adds at most n / 2^19 + 2^13
of them one after another, joined in some 40 steps: that many roundings of
2^-53. norm and the factor are rounded to fp32 once (2^-24), out once more to
its own type."""
import numpy as np
import pytest
import torch

import int4_weight_only_moe_amd as moe

pytestmark = pytest.mark.gpu

U, HALF_BF16 = 2.0 ** -24, 2.0 ** -8
BF16, F32 = torch.bfloat16, torch.float32


def make(sizes, kinds, seed, scale=0.01, shift=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for n, k in zip(sizes, kinds):
        room = torch.empty(n + shift, dtype=k, device="cuda")
        room[shift:] = (torch.randn(n, device="cuda", generator=g) * scale).to(k)
        out.append(room[shift:])
    return out


def check(grads, ratio, in_place=False):
    keep = [t.clone() for t in grads]
    want = sum(float(t.double().square().sum()) for t in grads)
    total = sum(t.numel() for t in grads)
    most = float(np.float32(ratio * want ** 0.5))
    out = grads if in_place else [torch.full_like(t, 7.0) for t in grads]
    s = moe.grad_sumsq(grads)
    assert abs(s.item() - want) <= (total / 2**19 + 2**13 + 40) * 2.0 ** -53 * want
    norm = moe.grad_clip(grads, s, most, out=None if in_place else out)
    root = s.item() ** 0.5
    whole = [t.clone() for t in keep]  # both in one call: the same sum in another order
    norm1 = moe.clip_grad_norm(whole, most)
    assert abs(norm1.item() - root) <= 1.01 * U * root + 2.0 ** -149
    assert all((a.double() - b.double()).abs().le((2.0 ** -7 if b.dtype == BF16 else 2.1 * U) * b.double().abs() + 2.0 ** -133).all()
               for a, b in zip(whole, out))
    assert norm.dtype == F32 and abs(norm.item() - root) <= U * root + 2.0 ** -149
    factor = most / root if root > most else 1.0
    for a, b in zip(keep, out):
        exact = a.double() * factor
        if factor == 1.0:
            assert torch.equal(a, b)
        else:
            half = HALF_BF16 if a.dtype == BF16 else U
            assert (b.double() - exact).abs().le((half + 1.01 * U) * exact.abs() + 2.0 ** -134 * (a.dtype == BF16) + 2.0 ** -149).all()
    if not in_place:
        assert all(torch.equal(a, b) for a, b in zip(keep, grads))
    return norm


@pytest.mark.parametrize("sizes", [(1,), (0,), (0, 3, 0), (8,), (2047,), (2048,), (2049,), (5000, 1, 2048, 0, 4096, 77),
                                   (100_000,), (2_000_003, 17), tuple([33] * 95), tuple([4097, 5] * 48), tuple([64] * 97),
                                   tuple([3000] * 300), tuple([100_001] * 300), (2048 * 2048, 2048 * 2048 + 1)])
def test_clip_sizes(sizes):
    mixed = [(F32, BF16)[i % 2] for i in range(len(sizes))]
    for kinds in ([F32] * len(sizes), [BF16] * len(sizes), mixed):
        for ratio in (0.25, 3.0):
            check(make(sizes, kinds, len(sizes)), ratio)
            check(make(sizes, kinds, len(sizes)), ratio, in_place=True)


def test_clip_unaligned():
    for shift in (1, 3):
        check(make((4099, 70_000, 5), (F32, BF16, F32), 4, shift=shift), 0.3)
        check(make((4099, 70_000, 5), (F32, BF16, BF16), 4, shift=shift), 0.3, in_place=True)
    g = make((5000,), (F32,), 5)
    s = moe.grad_sumsq(g)
    out = torch.zeros(5001, device="cuda")[1:]  # only the result is off a 16-byte border
    moe.grad_clip(g, s, 0.1, out=[out])
    want = [torch.empty_like(g[0])]
    moe.grad_clip(g, s, 0.1, out=want)
    assert torch.equal(out, want[0])


def test_clip_guard_bands():
    sizes = (1, 2049, 4095, 8)
    room = [torch.full((n + 32,), 5.0, device="cuda") for n in sizes]
    grads = make(sizes, (F32,) * 4, 6)
    moe.clip_grad_norm(grads, 0.01, out=[t[16:16 + n] for t, n in zip(room, sizes)])
    for t, n in zip(room, sizes):
        assert (t[:16] == 5).all() and (t[16 + n:] == 5).all() and (t[16:16 + n].abs() < 1).all()


def test_clip_magnitudes():
    """Squares beyond fp32's range, subnormal gradients, a norm of zero."""
    for scale in (1e30, 1e-30, 1e-40):
        check(make((5000, 300), (F32, BF16), 7, scale=scale), 0.5)
    # a factor below the smallest normal fp32 number: results of ordinary size keep their bits
    big = make((5000, 300), (F32, BF16), 7, scale=1e30)
    keep = [t.double() for t in big]
    root = sum(float(t.square().sum()) for t in keep) ** 0.5
    for most in (1e-10, 1e-13):
        out = [torch.empty_like(t) for t in big]
        moe.clip_grad_norm(big, most, out=out)
        for a, b in zip(keep, out):
            exact = a * (float(np.float32(most)) / root)
            half = HALF_BF16 if b.dtype == BF16 else U
            assert (b.double() - exact).abs().le((half + 2.1 * U) * exact.abs() + 2.0 ** -133 * (b.dtype == BF16) + 2.0 ** -148).all()
    zero = [torch.zeros(100, device="cuda")]
    assert moe.clip_grad_norm(zero, 0.0).item() == 0 and not zero[0].any()
    g = make((100,), (F32,), 8)
    keep = g[0].clone()
    moe.clip_grad_norm(g, float("inf"))
    assert torch.equal(g[0], keep)
    moe.clip_grad_norm(g, 0.0)
    assert not g[0].any()


@pytest.mark.parametrize("kind", (F32, BF16))
def test_clip_factors_far_below_the_normal_numbers(kind):
    """Gradients near fp32's largest value and bounds down to its smallest: factors to 2^-270, results of ordinary size."""
    grads = make((5000, 300), (kind, kind), 15, scale=3e37)
    keep = [t.double() for t in grads]
    root = sum(float(t.square().sum()) for t in keep) ** 0.5
    for most in (1e-15, 1e-20, 1e-22, 1e-25, 1e-30, 1e-35, 1e-40):
        out = [torch.full_like(t, 7.0) for t in grads]
        moe.clip_grad_norm(grads, most, out=out)
        assert most < 1e-29 or all(t.abs().max() > 0 for t in out)
        whole = [t.clone() for t in grads]
        moe.clip_grad_norm(whole, most)
        for a, b, c in zip(keep, out, whole):
            exact = a * (float(np.float32(most)) / root)
            half = HALF_BF16 if kind == BF16 else U
            assert (b.double() - exact).abs().le((half + 2.1 * U) * exact.abs() + 2.0 ** -133 * (kind == BF16) + 2.0 ** -148).all()
            assert torch.equal(b, c)


@pytest.mark.parametrize("bad", (float("nan"), float("inf"), -float("inf")))
def test_clip_not_finite_scales_nothing(bad):
    grads = make((3000, 50), (F32, BF16), 9)
    grads[0][2999] = bad
    keep = [t.clone() for t in grads]
    norm = moe.clip_grad_norm(grads, 1e-3)
    assert not torch.isfinite(norm).any()
    assert all(torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0)) for a, b in zip(keep, grads))


def test_clip_ranks_add_their_sums():
    a, b = make((700, 3000), (F32, F32), 10), make((5000,), (F32,), 11)
    both = moe.grad_sumsq(a) + moe.grad_sumsq(b)
    for part in (a, b):
        want = [t.double() * (0.1 / both.item() ** 0.5) for t in part]
        norm = moe.grad_clip(part, both, 0.1)
        assert abs(norm.item() - both.item() ** 0.5) <= U * norm.item()
        assert all((x.double() - y).abs().le(2.1 * U * y.abs()).all() for x, y in zip(part, want))


def test_clip_none():
    s = moe.grad_sumsq([], sumsq=torch.full((1,), 7.0, dtype=torch.float64, device="cuda"))
    assert s.item() == 0 and moe.grad_clip([], s, 1.0).item() == 0


def test_clip_the_same_gradient_twice():
    """An entry counts as often as it stands there; its results need memory of their own."""
    g = make((4000,), (F32,), 12)[0]
    s = moe.grad_sumsq([g, g])
    assert abs(s.item() - 2 * float(g.double().square().sum())) <= 1e-12 * s.item()
    out = [torch.empty_like(g), torch.empty_like(g)]
    moe.grad_clip([g, g], s, 0.1, out=out)
    assert torch.equal(out[0], out[1])
    for call in (lambda: moe.grad_clip([g, g], s, 0.1), lambda: moe.clip_grad_norm([g, g], 0.1)):
        with pytest.raises(moe.MoeError):
            call()


def test_clip_offsets_past_32_bits():
    n = 2**31 + 2**20 + 3
    big = torch.zeros(n, dtype=BF16, device="cuda")
    big[-5:] = 3.0
    big[0] = 4.0
    s = moe.grad_sumsq([big])
    assert s.item() == 16.0 + 45.0
    moe.grad_clip([big], s, 0.5 * 61.0 ** 0.5)
    assert big[-5:].tolist() == [1.5] * 5 and big[0].item() == 2.0 and big[-6].item() == 0


def test_clip_same_bits_streams_and_replays():
    sizes = (100_000, 7, 3000, 65_536) * 30
    grads = make(sizes, [F32, BF16] * 60, 13)
    keep = [t.clone() for t in grads]
    out = [torch.empty_like(t) for t in grads]
    ws = torch.empty(moe.moe_grad_norm_workspace_bytes(len(sizes)), dtype=torch.uint8, device="cuda")
    s, norm = torch.empty(1, dtype=torch.float64, device="cuda"), torch.empty(1, device="cuda")
    few, few_s, few_norm = [torch.empty_like(t) for t in grads[:60]], s.clone(), norm.clone()

    def call(stream=None):
        moe.grad_sumsq(grads, sumsq=s, workspace=ws, stream=stream)
        moe.grad_clip(grads, s, 0.5, out=out, norm=norm, stream=stream)
        moe.moe_clip_grad_norm(grads[:60], few, 0.4, ws, sumsq=few_s, norm=few_norm, stream=stream)
        return [s, norm, *out, *few, few_s, few_norm]

    first = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, call()))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for rep in range(4):
        for a, b in zip(grads, keep):
            a.copy_(b * (1 + rep % 2))
        for t in [s, norm, ws, *out, *few, few_s, few_norm]:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in (s, norm, *out, *few, few_s, few_norm)]
        assert all(torch.equal(a, b) for a, b in zip(replayed, call()))
        if rep % 2 == 0:
            assert all(torch.equal(a, b) for a, b in zip(replayed, first))


def test_clip_wrapper_refusals():
    g = make((8, 16), (F32, F32), 14)
    s = moe.grad_sumsq(g)
    for bad in (lambda: moe.grad_sumsq([g[0].half()]), lambda: moe.grad_sumsq([g[0], g[1].cpu()]),
                lambda: moe.grad_sumsq([torch.zeros((4, 4), device="cuda").t()]), lambda: moe.grad_sumsq([]),
                lambda: moe.grad_clip(g, s.float(), 1.0), lambda: moe.clip_grad_norm([], 1.0),
                lambda: moe.clip_grad_norm(g, 1.0, out=g[:1]), lambda: moe.grad_clip(g, s, 1.0, out=g[:1]),
                lambda: moe.grad_clip(g, s, 1.0, out=[g[1], g[0]]),
                lambda: moe.grad_clip(g, s, 1.0, out=[g[0], g[1].bfloat16()])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: moe.grad_clip(g, s, -1.0), lambda: moe.grad_clip([g[0], g[0][:4]], s, 1.0),
                lambda: moe.clip_grad_norm(g, float("nan"))):
        with pytest.raises(moe.MoeError):
            bad()
    with pytest.raises(moe.MoeError) as e:
        moe.grad_sumsq(g, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == moe.MOE_ERR_WORKSPACE
