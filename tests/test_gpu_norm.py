"""The norm with the residual's addition and its gradient against float64.

h, scales and 8-bit values are bit-exact: h is one rounding of a sum that fp32
holds well enough, and out8 is what the exact quotient rounds to. A bf16 result is
off by half a step (2^-8 relative) and the roundings of 2^-24 that come before
it: r carries 1, two products 1 each. Gradients count, per term: n = h r 1 (r is
given), u = w g exact, their product and the running sum over the lane's columns
(at most 32) and 6 + 4 + 15 to join lanes and waves, the mean 2, three more
steps; dw: the rows that one lane adds (at most M / 256, rounded up: of workgroups of
wide rows), 3 to join the waves of narrow rows, the rest is fp64."""
import itertools

import numpy as np
import pytest
import torch

import int4_weight_only_moe_amd as moe
import oracle

pytestmark = pytest.mark.gpu

U, HALF_BF16 = 2.0 ** -24, 2.0 ** -8
BF16, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.detach().double().cpu().numpy()


def tensors(M, N, dtype, seed, scale=3.0, gap=0, shift=0):
    """x, residual and weight; gap: columns between rows, shift: elements before the first."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, N, generator=g).to(BF16)
    res = (scale * torch.randn(M, N, generator=g) * torch.where(torch.rand(N, generator=g) < 0.05, 20.0, 1.0)).to(dtype)
    w = (1 + 0.3 * torch.randn(N, generator=g)).to(BF16)
    return placed(x, gap, shift), placed(res, gap, shift), w.cuda()


def placed(t, gap=0, shift=0):
    M, N = t.shape
    room = torch.full((M * (N + gap) + shift + gap,), 99.0, dtype=t.dtype, device="cuda")
    view = room[shift:shift + M * (N + gap)].view(M, N + gap)[:, :N]
    view.copy_(t)
    return view


def check(x, res, w, eps=1e-6, group=0, in_place=False, out=True, out_gap=0):
    first = x if x is not None else res
    M, N = first.shape
    dtype = BF16 if res is None else res.dtype
    h = x if res is None else res if x is None else (x.float() + res.float()).to(dtype)
    h = h.clone()
    bufs = moe.alloc_norm_buffers(M, N, dtype, out=out, rstd=True, quant_group=group)
    if out_gap:
        bufs.residual_out = placed(torch.zeros(M, N, dtype=dtype), out_gap, 1)
        bufs.out = placed(torch.zeros(M, N, dtype=BF16), out_gap, 1)
        if group:
            bufs.out8 = torch.zeros((M, N + out_gap), dtype=torch.uint8, device="cuda")[:, :N]
    if in_place:
        bufs.residual_out = first if res is None else res
    moe.add_rms_norm(x, w, bufs, residual=res, eps=eps)
    torch.cuda.synchronize()
    assert torch.equal(bufs.residual_out, h)
    y, r = oracle.rms_norm(f64(h), f64(w), eps)
    np.testing.assert_allclose(f64(bufs.rstd), r, rtol=2 * U)
    if out:
        err = np.abs(f64(bufs.out) - y)
        assert (err <= (HALF_BF16 + 4 * U) * np.abs(y) + 2.0 ** -134).all()
    if group:
        q, s = oracle.quantise(y, group)
        np.testing.assert_array_equal(bufs.scales.cpu().numpy(), s)
        got = bufs.out8.view(torch.float8_e4m3fn).float().cpu().numpy()
        np.testing.assert_array_equal(got, q.astype(np.float32))
    return bufs


WIDTHS = [1, 7, 8, 64, 127, 512, 520, 1000, 1024, 1025, 2048, 2056, 4096, 4100, 7168, 8192, 8200, 12345, 16384, 20000, 32768]


@pytest.mark.parametrize("N", WIDTHS)
def test_norm_widths(N):
    for i, (M, dtype) in enumerate(itertools.product((1, 5), (BF16, F32))):
        x, res, w = tensors(M, N, dtype, N + i)
        check(x, res, w)
        check(x, None, w)
        check(None, res, w, eps=0.5)
        check(x, res, w, group=N)
        for group in (32, 64, 128):
            if N % group == 0:
                check(x, res, w, group=group, out=i % 2 == 0)


@pytest.mark.parametrize("N,gap,shift,out_gap", [(64, 8, 0, 0), (64, 3, 0, 5), (512, 0, 1, 0), (7168, 24, 8, 8), (7168, 1, 3, 3),
                                                 (384, 128, 0, 128), (1000, 24, 0, 0), (2176, 5, 2, 7)])
def test_norm_strides_and_alignment(N, gap, shift, out_gap):
    for dtype in (BF16, F32):
        x, res, w = tensors(6, N, dtype, 60 + N, gap=gap, shift=shift)
        group = 64 if N % 64 == 0 else 0
        b = check(x, res, w, group=group, out_gap=out_gap)
        x2, res2, _ = tensors(6, N, dtype, 60 + N)
        a = check(x2, res2, w, group=group)
        assert torch.equal(a.rstd, b.rstd) or out_gap or gap or shift  # (the order of the sum depends on the layout)
        check(x, res, w, in_place=True)
        for view, room in ((x, gap), (res, gap)):  # what lies between the rows stays
            if room:
                whole = torch.as_strided(view, (6, room), (N + gap, 1), view.storage_offset() + N)
                assert (whole[:5] == 99).all()


def steps_apart(a, b):
    """Of positive fp32 values: the numbers of the type from one to the other."""
    return (a.view(torch.int32).long() - b.view(torch.int32).long()).abs().max().item()


@pytest.mark.parametrize("N", (64, 384, 1000, 2176, 7168, 16392))
def test_norm_layouts_agree(N):
    """The same rows contiguous and in other layouts. Rows of whole 16-byte chunks are added in the same order
    wherever they lie: the same bits. Others are added in another order, in fp64: rstd is at most the rounding of
    a neighbouring value."""
    for dtype in (BF16, F32):
        def run(gap, shift, out_gap):
            x, res, w = tensors(6, N, dtype, 60 + N, gap=gap, shift=shift)
            bufs = moe.alloc_norm_buffers(6, N, dtype, rstd=True, quant_group=N)
            if out_gap:
                bufs.residual_out = placed(torch.zeros(6, N, dtype=dtype), out_gap, out_gap)
                bufs.out = placed(torch.zeros(6, N, dtype=BF16), out_gap, out_gap)
                bufs.out8 = torch.zeros((6, N + out_gap), dtype=torch.uint8, device="cuda")[:, :N]
            return moe.add_rms_norm(x, w, bufs, residual=res)

        a = run(0, 0, 0)
        for layout in ((8, 0, 0), (0, 8, 0), (24, 16, 8), (0, 0, 16), (128, 0, 128)):
            b = run(*layout)
            assert torch.equal(a.rstd, b.rstd) and torch.equal(a.residual_out, b.residual_out), layout
            assert torch.equal(a.out, b.out) and torch.equal(a.scales, b.scales), layout
            assert torch.equal(a.out8.view(torch.uint8), b.out8.view(torch.uint8)), layout
        for layout in ((3, 0, 0), (0, 1, 0), (0, 0, 5), (24, 8, 3)):
            b = run(*layout)
            assert torch.equal(a.residual_out, b.residual_out), layout
            assert steps_apart(a.rstd, b.rstd) <= 1 and steps_apart(a.scales, b.scales) <= 1, layout
            # r one step apart, then the rounding to bf16 on both sides
            far = (a.out.double() - b.out.double()).abs()
            assert far.le((2 * HALF_BF16 + 4 * U) * a.out.double().abs() + 2.0 ** -133).all(), layout


def test_norm_many_rows_and_in_place():
    for N, M in ((256, 4099), (7168, 300)):
        x, res, w = tensors(M, N, BF16, N)
        check(x, res.clone(), w, in_place=True)
        bufs = moe.alloc_norm_buffers(M, N)
        want = moe.add_rms_norm(x, w, moe.alloc_norm_buffers(M, N), residual=res).out
        bufs.out = x  # the norm in place of x
        moe.add_rms_norm(x, w, bufs, residual=res)
        assert torch.equal(bufs.out, want)


def test_norm_empty_batch():
    w = torch.ones(64, dtype=BF16, device="cuda")
    bufs = moe.alloc_norm_buffers(0, 64, BF16, rstd=True, quant_group=32)
    x = torch.zeros((0, 64), dtype=BF16, device="cuda")
    moe.add_rms_norm(x, w, bufs, residual=x.clone())
    dh, dw = moe.add_rms_norm_backward(x, x.clone(), bufs.rstd, w)
    assert dh.shape == (0, 64) and not dw.any()


def test_norm_magnitudes():
    """Squares that over- and underflow fp32, subnormal rows, zero rows with and without eps."""
    N = 512
    g = torch.Generator().manual_seed(7)
    base = torch.randn(8, N, generator=g)
    scale = torch.tensor([1e30, 3e37, 1e-18, 1e-30, 1e-38, 1.0, 0.0, 1e-5])[:, None]
    w = (1 + 0.3 * torch.randn(N, generator=g)).to(BF16).cuda()
    for dtype in (BF16, F32):
        h = (base * scale).to(dtype).cuda()
        for eps in (0.0, 1e-6):
            rows = slice(0, 8) if eps else torch.tensor([0, 1, 2, 3, 5, 7])
            check(None, h[rows].contiguous(), w, eps=eps, group=64)
    zero = torch.zeros((2, N), dtype=BF16, device="cuda")
    bufs = check(None, zero, w, group=32)
    assert not bufs.out.any() and (bufs.scales == 2.0 ** -126).all() and not bufs.out8.view(torch.uint8).any()


def test_norm_beyond_the_range_of_rstd():
    """Without eps: r of rows below 2^-128 is infinite in fp32, other rows are not touched by it."""
    N = 256
    h = torch.ones((4, N), dtype=F32)
    h[0] *= 2.0 ** -140
    h[1] *= -(2.0 ** -120)
    h[2] = 0.0
    w = torch.ones(N, dtype=BF16, device="cuda")
    bufs = moe.alloc_norm_buffers(4, N, F32, rstd=True)
    moe.add_rms_norm(None, w, bufs, residual=h.cuda(), eps=0.0)
    assert torch.isinf(bufs.rstd[[0, 2]]).all() and bufs.rstd[1] == 2.0 ** 120 and bufs.rstd[3] == 1.0
    assert torch.isinf(bufs.out[0]).all() and (bufs.out[0] > 0).all() and torch.isnan(bufs.out[2]).all()
    assert (bufs.out[1] == -1.0).all() and (bufs.out[3] == 1.0).all()


def test_norm_nan_and_infinity():
    N = 256
    x, _, w = tensors(4, N, BF16, 9)
    x[1, 17], x[2, 200] = float("nan"), float("inf")
    for group in (0, 32, N):
        bufs = moe.alloc_norm_buffers(4, N, None, rstd=True, quant_group=group)
        moe.add_rms_norm(x, w, bufs)
        assert torch.isnan(bufs.out[1]).all() and torch.isnan(bufs.rstd[1])
        assert bufs.rstd[2] == 0 and torch.isnan(bufs.out[2, 200]) and not bufs.out[2, :200].any()
        assert torch.isfinite(bufs.out[[0, 3]].float()).all()
        if group:
            f = bufs.out8.float()
            assert torch.isnan(f[1]).all() and torch.isnan(bufs.scales[1]).all()
            assert torch.isnan(f[2, 200]) and torch.isnan(bufs.scales[2, -1 if group == N else 200 // 32])
            assert torch.isfinite(f[[0, 3]]).all()


def test_norm_8_bits_at_the_borders():
    """Rows whose quotients lie on or next to the middle between two e4m3 values:
    weights of 1, and a row's values whole multiples of its largest / 448 / 16."""
    rng = np.random.default_rng(10)
    M, N = 400, 256
    top = rng.integers(1, 256, (M, 1)) * 448 / 256
    h = rng.integers(-448 * 16, 448 * 16 + 1, (M, N)) / 16
    h[:, :1] = 448
    h = torch.from_numpy((h * top / 448).astype(np.float32))
    w = torch.ones(N, dtype=BF16, device="cuda")
    check(None, h.cuda(), w, group=N)
    check(None, h.to(BF16).cuda(), w, group=N)
    check(None, h.to(BF16).cuda(), w, group=32)
    k = torch.from_numpy((rng.integers(-240, 241, (M, N)) / 16).astype(np.float32))  # few distinct quotients
    k[:, 0] = 14.0
    check(None, k.to(BF16).cuda(), w, group=N, eps=0.0)


def check_backward(M, N, dtype, seed, passed=True, gap=0, shift=0, in_place=None, need_h=True):
    g = torch.Generator().manual_seed(seed)
    h = placed((3 * torch.randn(M, N, generator=g)).to(dtype), gap, shift)
    dy = placed((0.1 * torch.randn(M, N, generator=g)).to(BF16), gap, shift)
    dres = placed((0.1 * torch.randn(M, N, generator=g)).to(dtype), gap, shift) if passed else None
    w = (1 + 0.3 * torch.randn(N, generator=g)).to(BF16).cuda()
    r = torch.from_numpy(oracle.rms_norm(f64(h), f64(w), 1e-6)[1]).float().cuda()
    dh, dw, mag, wmag = oracle.rms_norm_backward(f64(dy), f64(h), f64(r), f64(w), f64(dres) if passed else None)
    to = {"dres": dres, "h": h, "dy": dy}.get(in_place)
    got, gw = moe.add_rms_norm_backward(dy, h, r, w, grad_residual=dres, need_h=need_h, grads=(to, None))
    if need_h:
        n = 1 + 1 + 32 + 25 + 2 + 3 + 1
        half = HALF_BF16 if dtype == BF16 else U
        err = np.abs(f64(got) - dh)
        assert (err <= n * U * mag + half * (np.abs(dh) + n * U * mag) + 2.0 ** -134).all()
    else:
        assert got is None
    err = np.abs(f64(gw) - dw)
    assert (err <= (-(-M // 256) + 3 + 1) * U * wmag + U * np.abs(dw) + 2.0 ** -149).all()
    return got, gw


@pytest.mark.parametrize("N", WIDTHS)
def test_norm_backward_widths(N):
    for i, (M, dtype) in enumerate(itertools.product((1, 6), (BF16, F32))):
        check_backward(M, N, dtype, N + i, passed=i % 2 == 0)
        check_backward(M, N, dtype, N + i, gap=3, shift=1)


def test_norm_backward_many_rows():
    for M, N in ((5000, 64), (1537, 1000), (1100, 2048), (513, 7168), (520, 2052)):
        check_backward(M, N, BF16, M)
        check_backward(M, N, F32, M, passed=False)


def test_norm_backward_in_place_and_parts():
    for N in (512, 4096):
        want = check_backward(40, N, BF16, 5)
        for where in ("dres", "h", "dy"):
            got = check_backward(40, N, BF16, 5, in_place=where)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        check_backward(40, N, F32, 6, in_place="dres")
        check_backward(40, N, F32, 6, passed=False, in_place="h")
        _, gw = check_backward(40, N, BF16, 5, passed=False, need_h=False)
        assert torch.equal(gw, want[1])
    h = torch.randn(8, 64, device="cuda", dtype=BF16)
    dh, dw = moe.add_rms_norm_backward(h, h, torch.ones(8, device="cuda"), h[0].contiguous(), need_weight=False)
    assert dw is None and dh.shape == (8, 64)


def test_norm_backward_nan_stays_in_its_row():
    N = 300  # the last lanes' columns lie past the end
    h, dy = torch.randn(5, N, device="cuda").to(BF16), torch.randn(5, N, device="cuda").to(BF16)
    h[2, 0] = float("nan")
    dy[3, 0] = float("inf")
    w = torch.ones(N, dtype=BF16, device="cuda")
    dh, _ = moe.add_rms_norm_backward(dy, h, torch.ones(5, device="cuda"), w)
    assert torch.isnan(dh[2]).all() and torch.isfinite(dh[[0, 1, 4]].float()).all()
    assert not torch.isfinite(dh[3].float()).any()


def test_norm_gradient_is_the_forwards_difference():
    """Against differences of the device's forward of an fp32 stream with all its bits in out8's place: rstd.
    d(sum r)/dh = -r^3 h / N; a gradient of the weight that picks r shows the same in the backward."""
    M, N, step = 3, 16, 2.0 ** -6
    g = torch.Generator().manual_seed(3)
    h = (torch.randn(M, N, generator=g) * 64).round().div(64).cuda()
    w = torch.ones(N, dtype=BF16, device="cuda")

    def norm_of(t):
        b = moe.alloc_norm_buffers(M, N, None, rstd=True)
        moe.add_rms_norm(None, w, b, residual=t)
        return b.rstd.double()[:, None] * t.double()  # n, before the bf16 rounding

    r = (norm_of(h)[:, :1] / h.double()[:, :1])[:, 0].float()
    dy = torch.randn(M, N, generator=g).to(BF16).cuda()
    dh, _ = moe.add_rms_norm_backward(dy, h, r, w)
    for c in range(N):
        up, down = h.clone(), h.clone()
        up[:, c] += step
        down[:, c] -= step
        d = ((norm_of(up) - norm_of(down)) * dy.double()).sum(1) / (2 * step)
        # third derivatives of n are below 3 r^3 (1 + |n|)^4 / N; rounding of rstd: 2 U |n| over the step
        n = norm_of(h).abs().max()
        tol = (step ** 2 / 6 * 3 * r.double().max() ** 3 * (1 + n) ** 4 / N + 2 * U * n / step) * dy.double().abs().sum(1) + 70 * U * 10
        assert (dh[:, c].double() - d).abs().le(tol).all()


def test_norm_same_bits_streams_and_replays():
    M, N = 200, 4096
    x, res, w = tensors(M, N, BF16, 20)
    keep = x.clone()
    bufs = moe.alloc_norm_buffers(M, N, BF16, rstd=True, quant_group=128)
    dy = torch.randn(M, N, device="cuda").to(BF16)
    ws = torch.empty(moe.moe_add_rms_norm_workspace_bytes(M, N), dtype=torch.uint8, device="cuda")
    grads = (torch.empty_like(x), torch.empty(N, device="cuda"))

    def call(stream=None):
        moe.add_rms_norm(x, w, bufs, residual=res, stream=stream)
        moe.add_rms_norm_backward(dy, bufs.residual_out, bufs.rstd, w, grads=grads, workspace=ws, stream=stream)
        return [bufs.residual_out, bufs.out, bufs.rstd, bufs.scales, bufs.out8.view(torch.uint8), *grads]

    first = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, call()))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = call()
    for rep in range(4):
        x.copy_(keep * (1 + rep % 2))
        for t in [*outs, ws]:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in outs]
        assert all(torch.equal(a, b) for a, b in zip(replayed, call()))
        if rep % 2 == 0:
            assert all(torch.equal(a, b) for a, b in zip(replayed, first))


def test_norm_more_rows_than_a_launch():
    """2^21 rows a launch; every output of the rows behind."""
    M, N = 2**21 + 70, 64
    x = torch.ones((M, N + 8), dtype=BF16, device="cuda")[:, :N]
    res = torch.zeros((M, N), device="cuda")
    g = torch.Generator().manual_seed(4)
    tail = slice(2**21 - 10, M)
    x[tail] = torch.randn(80, N, generator=g).to(BF16).cuda()
    res[tail] = torch.randn(80, N, generator=g).cuda()
    w = (1 + 0.3 * torch.randn(N, generator=g)).to(BF16).cuda()
    bufs = moe.add_rms_norm(x, w, moe.alloc_norm_buffers(M, N, F32, rstd=True, quant_group=32), residual=res)
    small = moe.add_rms_norm(x[tail], w, moe.alloc_norm_buffers(80, N, F32, rstd=True, quant_group=32), residual=res[tail])
    for name in ("residual_out", "out", "rstd", "scales"):
        assert torch.equal(getattr(bufs, name)[tail], getattr(small, name)), name
    assert torch.equal(bufs.out8[tail].view(torch.uint8), small.out8.view(torch.uint8))
    assert (bufs.residual_out[:2**21 - 10] == 1).all() and (bufs.rstd[:2**21 - 10] == bufs.rstd[0]).all()


def test_norm_workspace_of_a_larger_batch_and_offsets_past_32_bits():
    N = 1024
    M = 2**21 + 2**20 + 5  # M * N > 2^31 elements
    h = torch.ones((M, N), dtype=BF16, device="cuda")
    tail = torch.randn(64, N, generator=torch.Generator().manual_seed(2)).to(BF16)
    h[-64:] = tail.cuda()
    w = torch.ones(N, dtype=BF16, device="cuda")
    bufs = moe.alloc_norm_buffers(M, N, rstd=True, quant_group=128)
    moe.add_rms_norm(h, w, bufs)
    y, r = oracle.rms_norm(f64(tail), np.ones(N), 1e-6)
    assert (np.abs(f64(bufs.out[-64:]) - y) <= (HALF_BF16 + 4 * U) * np.abs(y)).all()
    q, s = oracle.quantise(y, 128)
    np.testing.assert_array_equal(bufs.out8[-64:].float().cpu().numpy(), q.astype(np.float32))
    ws = torch.empty(moe.moe_add_rms_norm_workspace_bytes(M, N), dtype=torch.uint8, device="cuda")
    dh, dw = moe.add_rms_norm_backward(bufs.out, h, bufs.rstd, w, workspace=ws)
    want, _, mag, _ = oracle.rms_norm_backward(f64(bufs.out[-64:]), f64(tail), f64(bufs.rstd[-64:]), np.ones(N))
    assert (np.abs(f64(dh[-64:]) - want) <= 65 * U * mag + HALF_BF16 * np.abs(want) + 65 * U * mag * HALF_BF16).all()
    small = moe.add_rms_norm_backward(bufs.out[-64:], h[-64:], bufs.rstd[-64:], w, workspace=ws)
    assert torch.equal(small[0], dh[-64:])


@pytest.mark.parametrize("M,N,dtype", [(2**24, 8, BF16), (2**20 + 5, 1000, F32), (2**20 + 77, 1028, BF16),
                                       (2**20 + 3, 2056, BF16), (2**19 + 1, 2056, F32), (2**18 + 9, 7001, BF16),
                                       (2**18 + 1, 16384, BF16), (2**18 + 3, 16392, BF16)])
def test_norm_weight_gradient_of_long_batches(M, N, dtype):
    """Terms of one sign, the same in most rows: what a running sum in fp32 loses over thousands of rows.
    The bound does not grow with M: n 1 rounding, 63 of the fp32 sum of a run of rows (the first is added to
    0), 1 for a wave's sum of its runs, 3 to join the waves of narrow rows, the rest is fp64, 1 for the result."""
    g = torch.Generator().manual_seed(N)
    h, dy = torch.empty((M, N), dtype=dtype, device="cuda"), torch.empty((M, N), dtype=BF16, device="cuda")
    h[:] = (0.5 + torch.rand(N, generator=g)).to(dtype).cuda()
    dy[:] = (0.5 + torch.rand(N, generator=g)).to(BF16).cuda()
    odd = torch.randint(0, M, (500,), generator=g).unique()  # some rows are others, the first and the last too
    odd = torch.cat([odd, torch.tensor([0, M - 1])]).unique().cuda()
    dy[odd] = (40 * torch.rand(len(odd), N, generator=g)).to(BF16).cuda()
    r = torch.full((M,), 0.7, device="cuda")
    r[odd] = (0.5 + torch.rand(len(odd), generator=g)).cuda()
    want = torch.zeros(N, dtype=torch.float64, device="cuda")
    for part in range(0, M, 2**16):
        rows = slice(part, part + 2**16)
        want += (dy[rows].double() * h[rows].double() * r[rows].double()[:, None]).sum(0)
    w = torch.ones(N, dtype=BF16, device="cuda")
    need = moe.moe_add_rms_norm_workspace_bytes(M, N)
    ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(2):  # (what the workspace holds does not matter)
        _, dw = moe.add_rms_norm_backward(dy, h, r, w, need_h=False, workspace=ws[:need])
        assert (dw.double() - want).abs().le((1 + 63 + 1 + 3 + 1) * U * want).all()
    assert (ws[need:] == 255).all()


@pytest.mark.parametrize("N,rows", [(40, 2**18), (1032, 2**15), (2056, 2**14), (16384, 2**14), (16392, 2**14)])
def test_norm_backward_around_the_longest_run(N, rows):
    """One row more than every lane's run of 64 holds, with a last workgroup that has only some of its rows."""
    for dtype in (BF16, F32):
        g = torch.Generator(device="cuda").manual_seed(N)
        M = rows + 3
        h = torch.randn((M, N), generator=g, device="cuda").to(dtype)
        dy = torch.randn((M, N), generator=g, device="cuda").to(BF16)
        r = 0.5 + torch.rand(M, generator=g, device="cuda")
        w = torch.randn(N, generator=g, device="cuda").to(BF16)
        some = moe.add_rms_norm_backward(dy[:100], h[:100], r[:100], w)[0]
        for m in (rows - 1, rows, rows + 1, rows + 3):
            dh, dw = moe.add_rms_norm_backward(dy[:m], h[:m], r[:m], w)
            assert torch.equal(dh[:100], some)
            t = dy[:m].double() * h[:m].double() * r[:m].double()[:, None]
            assert (dw.double() - t.sum(0)).abs().le((1 + 63 + 1 + 3 + 1) * U * t.abs().sum(0)).all()
            last = moe.add_rms_norm_backward(dy[m - 100:m], h[m - 100:m], r[m - 100:m], w)[0]
            assert torch.equal(dh[-100:], last)


def test_norm_backward_of_a_long_batch_replays():
    M, N = 2**14 + 40, 9000  # fp64 sums of more than 64 KB of LDS
    h, dy = torch.randn((M, N), device="cuda").to(BF16), torch.randn((M, N), device="cuda").to(BF16)
    keep, r, w = dy.clone(), 0.5 + torch.rand(M, device="cuda"), torch.randn(N, device="cuda").to(BF16)
    ws = torch.empty(moe.moe_add_rms_norm_workspace_bytes(M, N), dtype=torch.uint8, device="cuda")
    grads = (torch.empty_like(h), torch.empty(N, device="cuda"))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.add_rms_norm_backward(dy, h, r, w, grads=grads, workspace=ws)
    for rep in range(4):
        dy.copy_(keep * (1 + rep % 2))
        for t in (*grads, ws):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in grads]
        eager = moe.add_rms_norm_backward(dy, h, r, w)
        assert all(torch.equal(a, b) for a, b in zip(replayed, eager))


def test_norm_wrapper_refusals():
    x = torch.zeros((4, 64), dtype=BF16, device="cuda")
    w = torch.zeros(64, dtype=BF16, device="cuda")
    bufs = moe.alloc_norm_buffers(4, 64, BF16, rstd=True)
    for bad in (lambda: moe.add_rms_norm(x.float(), w, bufs), lambda: moe.add_rms_norm(x, w.float(), bufs),
                lambda: moe.add_rms_norm(x, w[:32], bufs), lambda: moe.add_rms_norm(x.t(), w, bufs),
                lambda: moe.add_rms_norm(x[:3], w, bufs), lambda: moe.add_rms_norm(None, w, bufs),
                lambda: moe.add_rms_norm(x, w, bufs, residual=x.half()),
                lambda: moe.add_rms_norm(x, w, bufs, residual=x.float()),  # residual_out is bf16
                lambda: moe.add_rms_norm(x.cpu(), w, bufs), lambda: moe.alloc_norm_buffers(4, 64, quant_group=48),
                lambda: moe.add_rms_norm_backward(x, x.half(), bufs.rstd, w),
                lambda: moe.add_rms_norm_backward(x, x, bufs.rstd[:3], w),
                lambda: moe.add_rms_norm_backward(x, x, bufs.rstd, w, grad_residual=x.float())):
        with pytest.raises(ValueError):
            bad()
    bufs.quant_group = 16
    bufs.out8, bufs.scales = torch.zeros((4, 64), dtype=torch.uint8, device="cuda"), torch.zeros((4, 4), device="cuda")
    with pytest.raises(moe.MoeError):
        moe.add_rms_norm(x, w, bufs)
    with pytest.raises(moe.MoeError) as e:
        moe.add_rms_norm_backward(x, x, bufs.rstd, w, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == moe.MOE_ERR_WORKSPACE
