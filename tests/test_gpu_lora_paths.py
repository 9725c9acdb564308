"""Low-rank adapters: sizes that take the kernels' less common ways, all
compared with float64 on the device.

Tolerances are counted as in test_gpu_lora.py; h and dh reach every result with
all their bits, so a result in bf16 adds its own half step, 2^-8, and nothing
else."""
import numpy as np
import pytest
import torch

import int4_weight_only_moe_amd as moe
from test_gpu_lora import Case, roundings

pytestmark = pytest.mark.gpu


def close(got, want, err, what):
    got = got.double()
    assert torch.isfinite(got).all(), what
    off = (got - want).abs()
    over = off - err - 1e-30
    assert (over <= 0).all(), (what, int((over > 0).sum()), float((off / (err + 1e-30)).max()))


def finite(t):
    """On the device in float64, with 0 where nothing is to be read."""
    return torch.nan_to_num(t.cuda().double(), nan=0.0, posinf=0.0, neginf=0.0)


def holds_block(ws, block):
    """Whether the workspace holds this [M, r] fp32 matrix, at any multiple of 256 bytes."""
    words = ws[: ws.numel() // 4 * 4].view(torch.int32)
    want = block.view(torch.int32).reshape(-1)
    at = torch.arange(0, words.numel() - want.numel() + 1, 64, device="cuda")
    at = at[(words[at] == want[0]) & (words[at + want.numel() - 1] == want[-1])]
    return any(torch.equal(words[i:i + want.numel()], want) for i in at.tolist())


def check(c, dx_base=True):
    """Forward with and without h, and backward; returns the forward call's workspace and h."""
    gids = torch.from_numpy(c.ids).cuda()
    x, a, b, s, base, dout = (getattr(c, n).cuda() for n in ("x", "a", "b", "scales", "base", "dout"))
    M, L, K, N, r = c.M, c.L, c.K, c.N, c.r
    half = 2.0 ** -24 if c.f32 else 2.0 ** -8
    none = torch.from_numpy(c.none).cuda()
    xx, aa, bb, gg, ss = finite(c.x), finite(c.a), finite(c.b), finite(c.dout), s.double()

    print(f"lora M={M} L={L} K={K} N={N} r={r} f32={c.f32} forward", flush=True)
    h = torch.full((M, r), 9.0, device="cuda")
    spaces = [torch.full((moe.moe_lora_workspace_bytes(M, L, K, N, r, back),), 0xFF, dtype=torch.uint8, device="cuda")
              for back in (False, False, True)]
    out = moe.lora_forward(x, gids, a, b, s, base=base, h=h, workspace=spaces[0])
    bare = moe.lora_forward(x, gids, a, b, s, base=base, workspace=spaces[1])
    assert torch.equal(out, bare)
    assert torch.equal(out[none], base[none]) and (h[none] == 0).all()
    for i in range(L):
        rows = (gids == i).nonzero()[:, 0]
        wh, mh = xx[rows] @ aa[i].T, xx[rows].abs() @ aa[i].abs().T
        close(h[rows], wh, mh * roundings(K), "h")
        want = base[rows].double() + ss[i] * (wh @ bb[i].T)
        err = ss[i] * (mh @ bb[i].abs().T) * (roundings(K) + roundings(r, 3) + 2.0 ** -24)
        err = err + half * (want.abs() + err) + 2.0 ** -24 * base[rows].double().abs()
        close(out[rows], want, err, "out")

    print("backward", flush=True)
    dxb = c.dx_base.cuda() if dx_base else None
    dx, da, db = moe.lora_backward(dout, x, gids, h, a, b, s, dx_base=dxb, workspace=spaces[2])
    zero = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    plus = dxb if dx_base else zero
    assert torch.equal(dx[none], plus[none])
    for i in range(L):
        rows = (gids == i).nonzero()[:, 0]
        dh, mdh = ss[i] * (gg[rows] @ bb[i]), ss[i] * (gg[rows].abs() @ bb[i].abs())
        edh = roundings(N, 3 if c.f32 else 1) + 2.0 ** -24
        want = plus[rows].double() + dh @ aa[i]
        err = (mdh @ aa[i].abs()) * (edh + roundings(r, 3))
        err = err + 2.0 ** -8 * (want.abs() + err) + 2.0 ** -24 * plus[rows].double().abs()
        close(dx[rows], want, err, "dx")
        close(da[i], dh.T @ xx[rows], (mdh.T @ xx[rows].abs()) * (edh + roundings(M, 3) + 2.0 ** -24), "da")
        hh = ss[i] * h[rows].double()
        close(db[i], gg[rows].T @ hh, (gg[rows].abs().T @ hh.abs()) * (2.0 ** -23 + roundings(M, 6 if c.f32 else 3)), "db")
    return spaces[1], h


@pytest.mark.parametrize("M,L,K,N,r,f32,ids", [
    (300, 3, 2048, 520, 64, False, "mixed"), (400, 2, 4096, 129, 32, True, "runs"), (700, 5, 1032, 264, 128, False, "mixed"),
    (1000, 4, 7168, 72, 48, False, "mixed"), (300, 2, 520, 60, 72, True, "mixed"), (257, 300, 768, 64, 64, False, "mixed"),
])
def test_lora_forward_sums_splits_once(M, L, K, N, r, f32, ids):
    """Grouped batches whose splits are added by a launch of their own: it leaves h
    in the workspace if the caller keeps none, with zeros for rows without an
    adapter, over partial sums that nothing wrote there."""
    c = Case(M, L, K, N, r, f32, ids, seed=70)
    ws, h = check(c)
    assert c.none.any() and holds_block(ws, h)


@pytest.mark.parametrize("M,L,K,N,r,f32", [
    (4100, 4, 7168, 72, 64, False), (1100, 2, 16384, 136, 64, False), (800, 2, 8192, 96, 64, True),
    (600, 1, 72, 7168, 64, True), (600, 3, 8200, 72, 128, False)])
def test_lora_long_contractions(M, L, K, N, r, f32):
    """Several steps of the contraction in each wave at ranks 64 and 128."""
    check(Case(M, L, K, N, r, f32, "runs", seed=71), dx_base=False)


@pytest.mark.parametrize("M,r,N,f32", [
    (26000, 8, 600, True), (26000, 32, 600, False), (26000, 64, 600, False), (26000, 64, 601, False), (17000, 64, 600, True),
    (9000, 128, 600, False), (9000, 128, 601, False), (9000, 128, 600, True), (9000, 72, 603, True)])
def test_lora_many_tiles_of_wide_rows(M, r, N, f32):
    """More tiles than workgroups that the chip holds, of rows of three column
    blocks: each wave of the expansion goes on to further columns, forward (N)
    and backward (K)."""
    check(Case(M, 3, 600, N, r, f32, "mixed", seed=72))


@pytest.mark.parametrize("r", range(8, 129, 8))
@pytest.mark.parametrize("M,f32", [(37, True), (150, False), (300, True), (520, False)])
def test_lora_every_rank(r, M, f32):
    check(Case(M, 3, 136, 72 if r % 16 else 75, r, f32, "mixed", seed=73))


def test_lora_many_rows_exact():
    """Tiles past 65535 of rows that have an adapter. All values are small whole
    numbers and every sum of magnitudes stays below 2^24, so every result is exact
    in any order (those in bf16 are at most 256): a tile left out or taken twice shows."""
    M, L, K, N, r = 4_300_000, 2, 8, 8, 8
    g = torch.Generator(device="cuda").manual_seed(5)

    def small(*shape):
        return torch.randint(-1, 2, shape, device="cuda", generator=g)

    x, dout, a, b = small(M, K), small(M, N), small(L, r, K), small(L, N, r)
    gids = torch.randint(0, L, (M,), device="cuda", generator=g, dtype=torch.int32)
    gids[torch.randint(0, M, (500,), device="cuda", generator=g)] = -1
    assert int((gids >= 0).sum()) > 64 * 65536 and bool((gids == L - 1).any())
    bf = torch.bfloat16
    h = torch.empty((M, r), device="cuda")
    base = torch.ones((M, N), device="cuda")
    out = moe.lora_forward(x.to(bf), gids, a.to(bf), b.to(bf), base=base, h=h)
    dx, da, db = moe.lora_backward(dout.float(), x.to(bf), gids, h, a.to(bf), b.to(bf))
    x, dout, a, b = x.double(), dout.double(), a.double(), b.double()
    for i in range(L):
        rows = (gids == i).nonzero()[:, 0]
        wh, dh = x[rows] @ a[i].T, dout[rows] @ b[i]
        assert torch.equal(h[rows].double(), wh)
        assert torch.equal(out[rows].double(), 1 + wh @ b[i].T)
        assert torch.equal(dx[rows].double(), dh @ a[i])
        for got, p, q in ((da[i], dh, x[rows]), (db[i], dout[rows], wh)):
            assert (p.abs().T @ q.abs()).max() < 2 ** 24
            assert torch.equal(got.double(), p.T @ q)
    none = (gids < 0).nonzero()[:, 0]
    assert (out[none] == 1).all() and (dx[none] == 0).all() and (h[none] == 0).all()
