"""Low-rank adapters of many requests, forward and backward, against the
float64 oracle.

Tolerances are bounds counted in roundings. A sum of n products of which the
matrix core adds 32 at a time takes at most n / 32 (times the parts of a
split factor) + 5 roundings inside one step + 24 to join waves, splits and
slots; each is at most 2^-23 of the sum of the terms' magnitudes (twice half
a step, as the matrix core need not round to nearest). A factor split into two
bf16 parts is off by 2^-17 of itself, one of three parts by nothing. A
result in bf16 adds half a step of it, 2^-8, one in fp32 2^-24."""
import numpy as np
import pytest
import torch

import int4_weight_only_moe_amd as moe
import oracle

pytestmark = pytest.mark.gpu

V = 2.0 ** -23


def roundings(n, parts=1):
    return (n / 32 * parts + 5 + 24) * V


def bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16)


class Case:
    def __init__(self, M, L, K, N, r, f32, ids="mixed", seed=0):
        rng = np.random.default_rng([seed, M, L, K, N, r])
        self.M, self.L, self.K, self.N, self.r, self.f32 = M, L, K, N, r, f32
        side = torch.float32 if f32 else torch.bfloat16
        self.x = bf16(rng.standard_normal((M, K)))
        self.a = bf16(rng.standard_normal((L, r, K)) * K ** -0.5)
        self.b = bf16(rng.standard_normal((L, N, r)) * r ** -0.5)
        self.scales = torch.from_numpy(rng.uniform(0.25, 2.0, L).astype(np.float32))
        self.base = torch.from_numpy(rng.standard_normal((M, N)).astype(np.float32)).to(side)
        self.dout = torch.from_numpy(rng.standard_normal((M, N)).astype(np.float32)).to(side)
        self.dx_base = bf16(rng.standard_normal((M, K)))
        if ids == "mixed":
            self.ids = rng.integers(0, L, M)
            self.ids[rng.random(M) < 0.15] = -1
            bad = rng.random(M) < 0.05
            self.ids[bad] = rng.choice([L, 2**31 - 1, -2**31], bad.sum())
        elif ids == "none":
            self.ids = np.full(M, -1)
        elif ids == "runs":
            self.ids = np.sort(rng.integers(-1, L, M))
        else:
            self.ids = np.full(M, int(ids))
        # rows without an adapter may hold anything on the input side
        none = (self.ids < 0) | (self.ids >= L)
        self.x[torch.from_numpy(none)] = float("nan")
        self.dout[torch.from_numpy(none)] = float("inf")
        # and so may an adapter that no row uses
        for i in set(range(L)) - set(self.ids.tolist()):
            self.a[i] = float("nan")
            self.b[i] = float("inf")
        self.none = none
        self.ids = self.ids.astype(np.int32)

    def clean(self):
        """Inputs as float64 arrays, with 0 where nothing is read."""
        z = lambda t: np.nan_to_num(t.double().numpy(), nan=0.0, posinf=0.0, neginf=0.0)  # noqa: E731
        return z(self.x), z(self.a), z(self.b), z(self.dout)


def forward_bounds(c, base):
    x, a, b, _ = c.clean()
    s = c.scales.double().numpy()
    out, h = oracle.lora_forward(x, c.ids, a, b, s, base)
    mag, hmag = oracle.lora_forward(np.abs(x), c.ids, np.abs(a), np.abs(b), s, np.zeros(base.shape))
    parts = 3 if c.f32 else 2
    herr = hmag * roundings(c.K)
    # mag = s |B| |A| |x|: h's error and the split's, and the expansion's sum over r
    err = mag * (roundings(c.K) + roundings(c.r, parts) + 2.0 ** -24 + (0 if c.f32 else 2.0 ** -17))
    half = 2.0 ** -24 if c.f32 else 2.0 ** -8
    err = err + half * (np.abs(out) + err) + 2.0 ** -24 * np.abs(base)
    return out, h, err, herr


def backward_bounds(c, h, dx_base):
    x, a, b, dout = c.clean()
    s = c.scales.double().numpy()
    dx, da, db = oracle.lora_backward(dout, x, c.ids, h, a, b, s, dx_base)
    mdx, mda, mdb = oracle.lora_backward(np.abs(dout), np.abs(x), c.ids, np.abs(h), np.abs(a), np.abs(b), s,
                                         np.zeros(dx_base.shape))
    parts = 3 if c.f32 else 1
    dh = roundings(c.N, parts) + 2.0 ** -24  # relative to |B| |dout|
    edx = mdx * (dh + roundings(c.r, 2) + 2.0 ** -17)
    edx = edx + 2.0 ** -8 * (np.abs(dx) + edx) + 2.0 ** -24 * np.abs(dx_base)
    eda = mda * (dh + roundings(c.M, 3) + 2.0 ** -24)
    edb = mdb * (2.0 ** -24 + roundings(c.M, 6 if c.f32 else 3) + 2.0 ** -24)
    return dx, da, db, edx, eda, edb


def within(got, want, err, what):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    off = np.abs(got - want)
    bad = off > err + 1e-30
    assert not bad.any(), (what, int(bad.sum()), float((off / (err + 1e-30)).max()))


SHAPES = [
    # M, L, K, N, rank, fp32 output side, ids
    (1, 1, 8, 1, 8, False, "0"), (1, 3, 256, 64, 16, False, "2"), (1, 2, 128, 7, 8, True, "1"),
    (2, 2, 24, 8, 8, False, "none"), (3, 2, 24, 7, 8, True, "mixed"), (16, 1, 64, 64, 32, False, "0"),
    (17, 4, 1032, 40, 24, False, "mixed"), (64, 64, 512, 256, 16, False, "mixed"),
    (65, 3, 128, 72, 16, False, "mixed"), (70, 2, 1024, 384, 128, True, "mixed"), (96, 5, 2048, 129, 64, False, "runs"),
    (130, 1, 512, 256, 64, False, "0"), (130, 2, 520, 1000, 40, False, "mixed"), (200, 300, 256, 133, 24, False, "mixed"),
    (257, 7, 136, 520, 128, False, "mixed"), (300, 2, 4096, 60, 8, True, "runs"), (512, 6, 256, 384, 32, True, "mixed"),
    (513, 1, 256, 264, 8, False, "mixed"), (600, 1024, 64, 40, 8, False, "mixed"), (1500, 9, 264, 200, 16, False, "runs"),
    (4200, 5, 64, 64, 32, False, "mixed"), (5000, 3, 128, 24, 64, True, "runs"),
]


@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_lora_matches_oracle(case):
    M, L, K, N, r, f32, ids = SHAPES[case]
    c = Case(M, L, K, N, r, f32, ids, seed=case)
    base = c.base.double().numpy()
    out, h, err, herr = forward_bounds(c, base)
    d = {n: getattr(c, n).cuda() for n in ("x", "a", "b", "scales", "base", "dout", "dx_base")}
    gids = torch.from_numpy(c.ids).cuda()
    print(f"lora {SHAPES[case]} forward", flush=True)
    gh = torch.full((M, r), 9.0, device="cuda")
    ws = torch.full((moe.moe_lora_workspace_bytes(M, L, K, N, r, False),), 0xFF, dtype=torch.uint8, device="cuda")
    got = moe.lora_forward(d["x"], gids, d["a"], d["b"], d["scales"], base=d["base"], h=gh, workspace=ws)
    torch.cuda.synchronize()
    within(gh, h, herr, "h")
    within(got, out, err, "out")
    none = torch.from_numpy(c.none).cuda()
    assert torch.equal(got[none], d["base"][none]) and (gh[none] == 0).all()

    print("backward", flush=True)
    hh = gh.double().cpu().numpy()
    dxb = c.dx_base.double().numpy()
    dx, da, db, edx, eda, edb = backward_bounds(c, hh, dxb)
    ws = torch.full((moe.moe_lora_workspace_bytes(M, L, K, N, r, True),), 0xFF, dtype=torch.uint8, device="cuda")
    gdx, gda, gdb = moe.lora_backward(d["dout"], d["x"], gids, gh, d["a"], d["b"], d["scales"], dx_base=d["dx_base"],
                                      workspace=ws)
    torch.cuda.synchronize()
    within(gdx, dx, edx, "dx")
    within(gda, da, eda, "da")
    within(gdb, db, edb, "db")
    assert torch.equal(gdx[none], d["dx_base"][none])


@pytest.mark.parametrize("f32,N", [(False, 72), (True, 60), (False, 37)])
def test_lora_strides_in_place_and_no_base(f32, N):
    """Column slices of wider matrices; out = base; no base; no scales; nothing else is written."""
    M, L, K, r = 150, 3, 96, 16
    c = Case(M, L, K, N, r, f32, "mixed", seed=50)
    gids, a, b = torch.from_numpy(c.ids).cuda(), c.a.cuda(), c.b.cuda()
    plain = moe.lora_forward(c.x.cuda(), gids, a, b, c.scales.cuda(), base=c.base.cuda())
    wide_x = torch.full((M, K + 32), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide_x[:, 16:16 + K] = c.x.cuda()
    x = wide_x[:, 16:16 + K]
    for lead in (16, 3):  # 16-byte aligned rows, and rows that are not
        wide = torch.full((M, N + 24), 3.5, dtype=c.base.dtype, device="cuda")
        wide[:, lead:lead + N] = c.base.cuda()
        out = wide[:, lead:lead + N]
        assert moe.lora_forward(x, gids, a, b, c.scales.cuda(), base=out, out=out) is out
        assert torch.equal(out, plain), lead
        assert (wide[:, :lead] == 3.5).all() and (wide[:, lead + N:] == 3.5).all()
    none = torch.from_numpy(c.none).cuda()
    o2 = torch.full_like(plain, 5.0)
    moe.lora_forward(x, gids, a, b, base=None, out=o2)
    c.scales = torch.ones(L)
    want, _, err, _ = forward_bounds(c, np.zeros((M, N)))
    within(o2, want, err, "no base, no scales")
    assert (o2[none] == 0).all()

    # backward on the same slices
    h = torch.zeros((M, r), device="cuda")
    moe.lora_forward(x, gids, a, b, base=None, out=o2, h=h)
    wide_g = torch.full((M, N + 24), float("nan"), dtype=c.base.dtype, device="cuda")
    wide_g[:, 3:3 + N] = c.dout.cuda()
    wide_dx = torch.full((M, K + 32), 2.5, dtype=torch.bfloat16, device="cuda")
    wide_dx[:, 8:8 + K] = c.dx_base.cuda()
    dxv = wide_dx[:, 8:8 + K]
    grads = (dxv, torch.empty(a.shape, device="cuda"), torch.empty(b.shape, device="cuda"))
    moe.lora_backward(wide_g[:, 3:3 + N], x, gids, h, a, b, dx_base=dxv, grads=grads)
    one = moe.lora_backward(c.dout.cuda(), c.x.cuda(), gids, h, a, b, dx_base=c.dx_base.cuda())
    for p, q in zip(grads, one):
        assert torch.equal(p, q)
    assert (wide_dx[:, :8] == 2.5).all() and (wide_dx[:, 8 + K:] == 2.5).all()
    # without dx, and dx without a base
    none_dx = moe.lora_backward(c.dout.cuda(), c.x.cuda(), gids, h, a, b, need_dx=False)
    assert none_dx[0] is None and torch.equal(none_dx[1], one[1]) and torch.equal(none_dx[2], one[2])
    z = moe.lora_backward(c.dout.cuda(), c.x.cuda(), gids, h, a, b)
    z0 = moe.lora_backward(c.dout.cuda(), c.x.cuda(), gids, h, a, b, dx_base=torch.zeros_like(c.dx_base).cuda())
    assert torch.equal(z[0], z0[0])


def test_lora_offsets_past_32_bits():
    """Rows whose element offset passes 2^31 in x and in the output."""
    M, K, N, r, wide = 80, 64, 32, 8, 28_000_000
    c = Case(M, 2, K, N, r, False, "mixed", seed=51)
    room = torch.empty((M, wide), dtype=torch.bfloat16, device="cuda")  # 4.5 GB
    assert (M - 1) * wide > 2**31
    room[:, :K] = c.x.cuda()
    room[:, 512:512 + N] = c.base.cuda()
    gids, a, b, s = torch.from_numpy(c.ids).cuda(), c.a.cuda(), c.b.cuda(), c.scales.cuda()
    out = room[:, 512:512 + N]
    h = torch.empty((M, r), device="cuda")
    moe.lora_forward(room[:, :K], gids, a, b, s, base=out, out=out, h=h)
    assert torch.equal(out, moe.lora_forward(c.x.cuda(), gids, a, b, s, base=c.base.cuda()))
    room[:, 512:512 + N] = c.dout.cuda()
    room[:, 1024:1024 + K] = c.dx_base.cuda()
    dxv = room[:, 1024:1024 + K]
    grads = (dxv, torch.empty(a.shape, device="cuda"), torch.empty(b.shape, device="cuda"))
    moe.lora_backward(out, room[:, :K], gids, h, a, b, s, dx_base=dxv, grads=grads)
    want = moe.lora_backward(c.dout.cuda(), c.x.cuda(), gids, h, a, b, s, dx_base=c.dx_base.cuda())
    assert all(torch.equal(p, q) for p, q in zip(grads, want))


def test_lora_of_no_rows():
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    ids = torch.empty(0, dtype=torch.int32, device="cuda")
    a = torch.randn((2, 8, 64), device="cuda").to(torch.bfloat16)
    b = torch.randn((2, 16, 8), device="cuda").to(torch.bfloat16)
    assert moe.lora_forward(x, ids, a, b).shape == (0, 16)
    grads = (x, torch.full(a.shape, 4.0, device="cuda"), torch.full(b.shape, 4.0, device="cuda"))
    moe.lora_backward(torch.empty((0, 16), device="cuda"), x, ids, torch.empty((0, 8), device="cuda"), a, b, grads=grads)
    assert (grads[1] == 0).all() and (grads[2] == 0).all()


@pytest.mark.parametrize("M", [5, 700])
def test_lora_same_bits_streams_and_replays(M):
    L, K, N, r = 4, 256, 136, 16
    c = Case(M, L, K, N, r, False, "mixed", seed=52)
    other = Case(M, L, K, N, r, False, "runs", seed=53)
    x, a, b, s, base, dout = (getattr(c, n).cuda() for n in ("x", "a", "b", "scales", "base", "dout"))
    gids = torch.from_numpy(c.ids).cuda()
    # every adapter has finite weights here: the graph is replayed on other ids
    a, b = torch.nan_to_num(a), torch.nan_to_num(b, posinf=0.0)
    h = torch.zeros((M, r), device="cuda")
    out = torch.empty_like(base)
    grads = (torch.empty_like(x), torch.empty(a.shape, device="cuda"), torch.empty(b.shape, device="cuda"))

    def call(stream=None):
        moe.lora_forward(x, gids, a, b, s, base=base, out=out, h=h, stream=stream)
        moe.lora_backward(dout, x, gids, h, a, b, s, grads=grads, stream=stream)
        return [t.clone() for t in (out, h, *grads)]

    first = call()
    assert all(torch.equal(p, q) for p, q in zip(first, call()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = call()
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, again))
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)  # buffers of this stream, work on the other
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, (out, h, *grads)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.lora_forward(x, gids, a, b, s, base=base, out=out, h=h)
        moe.lora_backward(dout, x, gids, h, a, b, s, grads=grads)
    for rep in range(4):
        new = c if rep % 2 == 0 else other
        gids.copy_(torch.from_numpy(new.ids).cuda())
        x.copy_(new.x.cuda())
        dout.copy_(new.dout.cuda())
        for t in (out, h, *grads):
            t.fill_(-1.0)
        g.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in (out, h, *grads)]
        assert all(torch.equal(p, q) for p, q in zip(replayed, call())), rep
        if rep % 2 == 0:
            assert all(torch.equal(p, q) for p, q in zip(replayed, first))


def test_lora_wrapper_refusals():
    bf = torch.bfloat16
    x = torch.zeros((4, 64), dtype=bf, device="cuda")
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    a = torch.zeros((2, 8, 64), dtype=bf, device="cuda")
    b = torch.zeros((2, 16, 8), dtype=bf, device="cuda")
    f = moe.lora_forward
    out = torch.zeros((4, 16), dtype=bf, device="cuda")
    for bad in (lambda: f(x.float(), ids, a, b), lambda: f(x, ids.long(), a, b), lambda: f(x, ids[:3], a, b),
                lambda: f(x, ids, a.float(), b), lambda: f(x, ids, a, b[:1]), lambda: f(x, ids, a, b[:, :, :7]),
                lambda: f(x, ids, a, b, scales=torch.ones(3, device="cuda")), lambda: f(x.cpu(), ids, a, b),
                lambda: f(x, ids.cpu(), a, b), lambda: f(x, ids, a, b, base=out.float(), out=out),
                lambda: f(x, ids, a, b, out=out.half()), lambda: f(x, ids, a, b, out=out.t().contiguous().t()),
                lambda: f(x, ids, a, b, h=torch.zeros((4, 7), device="cuda")),
                lambda: f(x[:, :60], ids, a[:, :, :60].contiguous(), b),
                lambda: moe.lora_backward(out, x, ids, torch.zeros((4, 8), device="cuda", dtype=bf), a, b)):
        with pytest.raises(ValueError):
            bad()
    ws = torch.zeros(64, dtype=torch.uint8, device="cuda")
    for call, status in ((lambda: f(x, ids, a, b, workspace=ws), moe.MOE_ERR_WORKSPACE),
                         (lambda: f(torch.zeros((4, 65), dtype=bf, device="cuda")[:, :64], ids, a, b), moe.MOE_ERR_INVALID_ARG),
                         (lambda: f(x[:1].expand(4, 64), ids, a, b), moe.MOE_ERR_INVALID_ARG)):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.status == status


def test_lora_many_rows():
    """More tiles than a grid's second dimension holds (M / 64 > 65535)."""
    M, L, K, N, r = 4_300_000, 2, 8, 8, 8
    rng = np.random.default_rng(3)
    x = torch.randn((M, K), device="cuda").to(torch.bfloat16)
    a = bf16(rng.standard_normal((L, r, K))).cuda()
    b = bf16(rng.standard_normal((L, N, r))).cuda()
    gids = torch.randint(-1, L, (M,), device="cuda", dtype=torch.int32)
    h = torch.empty((M, r), device="cuda")
    base = torch.zeros((M, N), device="cuda")
    out = moe.lora_forward(x, gids, a, b, base=base, h=h)
    dx, da, db = moe.lora_backward(out, x, gids, h, a, b)
    rows = torch.cat([torch.arange(1000), torch.arange(M - 1000, M)]).cuda()
    c = Case(2000, L, K, N, r, True, "mixed")  # the bounds of a small case with these rows
    c.x, c.a, c.b, c.ids, c.scales = x[rows].cpu(), a.cpu(), b.cpu(), gids[rows].cpu().numpy(), torch.ones(L)
    want, wh, err, herr = forward_bounds(c, np.zeros((2000, N)))
    within(out[rows], want, err, "out")
    within(h[rows], wh, herr, "h")
    for i in range(L):  # the sums over all rows, in fp64 on the device
        m = gids == i
        hs = h[m].double()
        wb = out[m].double().t() @ hs
        mag = out[m].double().abs().t() @ hs.abs()
        assert ((db[i].double() - wb).abs() <= mag * (roundings(M, 6) + 2.0 ** -23)).all()
        assert torch.isfinite(da[i]).all()
    assert torch.isfinite(dx.float()).all()


def test_lora_reused_workspace():
    """One workspace of the largest batch, backward, serves smaller ones and forward calls."""
    L, K, N, r = 5, 136, 96, 24
    ws = torch.empty(moe.moe_lora_workspace_bytes(3000, L, K, N, r, True), dtype=torch.uint8, device="cuda")
    for M in (3000, 1, 257, 900, 64):
        c = Case(M, L, K, N, r, False, "mixed", seed=60)
        d = {n: getattr(c, n).cuda() for n in ("x", "a", "b", "scales", "base", "dout")}
        gids = torch.from_numpy(c.ids).cuda()
        h, h2 = torch.empty((M, r), device="cuda"), torch.empty((M, r), device="cuda")
        one = moe.lora_forward(d["x"], gids, d["a"], d["b"], d["scales"], base=d["base"], h=h, workspace=ws)
        two = moe.lora_forward(d["x"], gids, d["a"], d["b"], d["scales"], base=d["base"], h=h2)
        assert torch.equal(one, two) and torch.equal(h, h2)
        g1 = moe.lora_backward(d["dout"], d["x"], gids, h, d["a"], d["b"], d["scales"], workspace=ws)
        g2 = moe.lora_backward(d["dout"], d["x"], gids, h, d["a"], d["b"], d["scales"])
        assert all(torch.equal(p, q) for p, q in zip(g1, g2))


def test_lora_backward_larger_than_the_cache():
    """Ten times the rows of one case, with more than 256 MB to move: the same
    dx for each repetition (with a base, in place, and without one), ten times
    the weight gradients."""
    M, L, K, N, r, times = 230, 3, 20480, 72, 16, 10
    assert times * M * (6 * K + 2 * N) > 2**28 > M * (6 * K + 2 * N)
    c = Case(M, L, K, N, r, False, "mixed", seed=61)
    gids, a, b, s = torch.from_numpy(c.ids).cuda(), c.a.cuda(), c.b.cuda(), c.scales.cuda()
    x, dout, dxb = c.x.cuda(), c.dout.cuda(), c.dx_base.cuda()
    h = torch.empty((M, r), device="cuda")
    moe.lora_forward(x, gids, a, b, s, h=h)
    dx, da, db, edx, eda, edb = backward_bounds(c, h.double().cpu().numpy(), c.dx_base.double().numpy())
    many = [t.repeat(times, *[1] * (t.dim() - 1)) for t in (dout, x, gids, h, dxb)]
    got = moe.lora_backward(*many[:4], a, b, s, dx_base=many[4])
    for i in range(times):
        within(got[0][i * M:(i + 1) * M], dx, edx, "dx")
    # eda and edb hold roundings(M, 3) of the terms' magnitudes; the longer sums take the difference more
    more = (roundings(times * M, 3) - roundings(M, 3)) / roundings(M, 3)
    within(got[1], times * da, times * eda * (1 + more), "da")
    within(got[2], times * db, times * edb * (1 + more), "db")
    place = many[4].clone()
    moe.lora_backward(*many[:4], a, b, s, dx_base=place, grads=(place, *[torch.empty_like(t) for t in got[1:]]))
    assert torch.equal(place, got[0])
    bare = moe.lora_backward(*many[:4], a, b, s)
    zero = moe.lora_backward(*many[:4], a, b, s, dx_base=torch.zeros_like(place))
    assert torch.equal(bare[0], zero[0])


@pytest.mark.parametrize("r", [8, 16, 32, 40, 64, 72, 128])
@pytest.mark.parametrize("f32", [False, True])
def test_lora_expansion_keeps_all_bits(r, f32):
    """h (forward) and dh (backward) reach the result with all 24 bits of fp32,
    whatever the result's type. Three ranks hold v = p1 + p2 + p3 (three bf16
    numbers of 8 bits each, so v has 24), -p1 and -p2, and the other weights make
    every column their sum, p3. All terms are multiples of p3's last bit u, and any
    of them add up to less than 2^24 u, so no order of the additions rounds: the
    result is p3 exactly. With the last 8 bits of v lost it would be 0."""
    M, K, N, L = 150, 64, 40, 3
    rng = np.random.default_rng(r)
    u = 2.0 ** -20
    p3 = rng.integers(64, 128, M) * rng.choice([-1.0, 1.0], M) * u
    p2 = rng.integers(64, 127, M) * 2.0 ** 8 * u
    p1 = rng.integers(64, 127, M) * 2.0 ** 16 * u
    pieces = np.stack([p1, p2, p3], 1)
    assert (np.abs(pieces).sum(1) < 2.0 ** 24 * u).all()
    ids = torch.from_numpy((np.arange(M) % L).astype(np.int32)).cuda()
    mix = np.array([[1.0, 1.0, 1.0], [-1.0, 0.0, 0.0], [0.0, -1.0, 0.0]])  # the three ranks' values of the pieces
    side = torch.float32 if f32 else torch.bfloat16

    x, a, b = np.zeros((M, K)), np.zeros((L, r, K)), np.zeros((L, N, r))
    x[:, :3], a[:, r - 3:, :3], b[:, :, r - 3:] = pieces, mix, 1.0
    h = torch.empty((M, r), device="cuda")
    out = moe.lora_forward(bf16(x).cuda(), ids, bf16(a).cuda(), bf16(b).cuda(),
                           base=torch.zeros((M, N), dtype=side, device="cuda"), h=h)
    np.testing.assert_array_equal(h.double().cpu().numpy()[:, r - 3:], pieces @ mix.T)
    np.testing.assert_array_equal(out.double().cpu().numpy(), np.repeat(p3[:, None], N, 1))

    g, a, b = np.zeros((M, N)), np.zeros((L, r, K)), np.zeros((L, N, r))
    g[:, :3], b[:, :3, r - 3:], a[:, r - 3:] = pieces, mix.T, 1.0
    dx, _, _ = moe.lora_backward(torch.from_numpy(g).to(side).cuda(), bf16(x).cuda(), ids, h, bf16(a).cuda(),
                                 bf16(b).cuda())
    np.testing.assert_array_equal(dx.double().cpu().numpy(), np.repeat(p3[:, None], K, 1))


def test_lora_backward_buffers_and_need_dx():
    """need_dx decides about dx, whatever buffers the caller passes: one that is there is left
    as it was without it, one that is missing is allocated with it."""
    M, L, K, N, r = 40, 2, 64, 48, 8
    c = Case(M, L, K, N, r, False, "mixed", seed=62)
    gids, x, a, b, dout = torch.from_numpy(c.ids).cuda(), c.x.cuda(), c.a.cuda(), c.b.cuda(), c.dout.cuda()
    h = torch.empty((M, r), device="cuda")
    moe.lora_forward(x, gids, a, b, h=h)
    want = moe.lora_backward(dout, x, gids, h, a, b)
    kept = (torch.full_like(x, 7.0), torch.zeros_like(want[1]), torch.zeros_like(want[2]))
    got = moe.lora_backward(dout, x, gids, h, a, b, need_dx=False, grads=kept)
    assert got[0] is None and got[1] is kept[1] and got[2] is kept[2] and (kept[0] == 7.0).all()
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    more = moe.lora_backward(dout, x, gids, h, a, b, grads=got)  # those of a call without dx
    assert torch.equal(more[0], want[0]) and more[1] is kept[1] and more[2] is kept[2]
    again = moe.lora_backward(dout, x, gids, h, a, b, grads=kept)
    assert all(p is q for p, q in zip(again, kept)) and torch.equal(kept[0], want[0])


@pytest.mark.parametrize("swap", [False, True])
def test_lora_weight_gradient_keeps_all_bits(swap):
    """grad_b of fp32 gradients: u v with u = 1 + 2^-8 (two bf16 parts) and
    v = 1 + 2^-8 - 2^-17 (three), in either role. Further rows take every product
    of their parts away again but the one of the smaller parts, -2^-25, which fp32
    holds beside nothing else: all terms are multiples of it, and what is left of
    each pair of parts is below 2^-6."""
    u, v = (1.0, 2.0 ** -8), (1.0, 2.0 ** -8, -2.0 ** -17)
    rows = [(sum(u), sum(v))] + [(-p, q) for p in u for q in v if (p, q) != (u[1], v[2])]
    if swap:
        rows = [(q, p) for p, q in rows]
    M, L, K, N, r = len(rows), 1, 64, 40, 16
    side = torch.tensor(rows, dtype=torch.float64)
    assert (side.float().double() == side).all()
    dout = side[:, :1].float().expand(M, N).contiguous().cuda()
    h = side[:, 1:].float().expand(M, r).contiguous().cuda()
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    _, _, db = moe.lora_backward(dout, z(M, K), torch.zeros(M, dtype=torch.int32, device="cuda"), h, z(L, r, K), z(L, N, r))
    assert (db == -2.0 ** -25).all()
