"""Host-side checks of the entry points between the layer and the rest of a
model (no GPU): sizes, statuses before any launch, overlaps of clipped gradients,
and extreme sizes in a build of the host code with the sanitizers."""
import ctypes
import os
import shutil
import subprocess

import pytest

import int4_weight_only_moe_amd as moe
from int4_weight_only_moe_amd import build as b
from test_abi_sanitize import CLANG, SANITIZE_HOST, _run

P = 0x10000  # an aligned non-null address; validation fails before any use
ARG, UNS, WS, CAP, OK = (moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE, moe.MOE_ERR_CAPACITY,
                         moe.MOE_OK)


def route(M=4, E=64, k=4, scoring=1, bias=P, G=8, top=4, each=2, scale=1.0, valid=None, bm=16, logits=P, ids=P, w=P,
          rows=P, blocks=P, off=P, npp=P, cap=None):
    if cap is None:
        cap = moe.moe_route_align_capacity(max(M, 0), E, k, bm)
    return moe.lib().moe_route_scored(logits, M, E, k, scoring, bias, G, top, each, 1, scale, valid, bm, ids, w, rows,
                                      blocks, off, npp, cap, None)


def test_route_scored_validation():
    assert route(M=0, logits=None, ids=None, w=None) == OK
    assert route(M=0, logits=None, ids=None, w=None, rows=None, blocks=None, off=None, npp=None, bm=7) == OK
    for bad in (dict(M=-1), dict(E=0), dict(k=0), dict(scoring=2), dict(scoring=-1), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(G=0), dict(top=0), dict(top=9), dict(each=0), dict(each=3),
                dict(logits=None), dict(ids=None), dict(w=None), dict(rows=None), dict(blocks=None), dict(off=None),
                dict(npp=None), dict(logits=P + 2), dict(bias=P + 1), dict(ids=P + 2), dict(w=P + 2), dict(rows=P + 1),
                dict(npp=P + 2), dict(off=P + 2), dict(blocks=P + 2)):
        assert route(**bad) == ARG, bad
    for bad in (dict(E=1025), dict(k=17), dict(E=4, k=5, G=1, top=1, cap=64), dict(G=7), dict(G=65, E=65 * 8), dict(bm=17),
                dict(G=64, top=64), dict(top=1, G=32), dict(M=1 << 28)):
        assert route(**{"cap": 1 << 40, **bad}) == UNS, bad  # (G = 64: groups of one expert have no two highest)
    assert route(cap=moe.moe_route_align_capacity(4, 64, 4, 16) - 16) == CAP
    assert route(cap=moe.moe_route_align_capacity(4, 64, 4, 16) + 8) == CAP


def test_route_scored_backward_validation():
    def call(M=4, E=8, k=2, scoring=0, scale=1.0, logits=P, ids=P, gw=P, base=P, grad=P):
        return moe.lib().moe_route_scored_backward(logits, M, E, k, scoring, 1, scale, ids, gw, base, grad, None)

    assert call(M=0, logits=None, ids=None, gw=None, grad=None) == OK
    for bad in (dict(M=-1), dict(E=0), dict(k=0), dict(scoring=3), dict(scale=float("nan")), dict(logits=None),
                dict(ids=None), dict(gw=None), dict(grad=None), dict(logits=P + 2), dict(ids=P + 1), dict(gw=P + 2),
                dict(base=P + 2), dict(grad=P + 1)):
        assert call(**bad) == ARG, bad
    assert call(E=1025) == UNS and call(k=9) == UNS and call(E=64, k=17) == UNS and call(M=1 << 29) == UNS


def norm(M=4, N=256, x=P, ldx=256, res=P + 4096, ldr=256, kind=0, w=P, eps=1e-6, ro=P + 8192, ldro=256, out=P + 16384,
         ldo=256, o8=None, ld8=256, sc=None, group=0, rstd=None):
    return moe.lib().moe_add_rms_norm(x, ldx, res, ldr, kind, M, N, w, eps, ro, ldro, out, ldo, o8, ld8, sc, group, rstd,
                                      None)


def test_norm_validation():
    assert norm(M=0, x=None, res=None, w=None, out=None) == OK
    for bad in (dict(M=-1), dict(N=0), dict(kind=2), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
                dict(x=None, res=None), dict(res=None, kind=1), dict(w=None), dict(out=None), dict(ldx=255),
                dict(ldr=200), dict(ldro=0), dict(ldo=255), dict(x=P + 1), dict(res=P + 2, kind=1), dict(ro=P + 2, kind=1),
                dict(out=P + 1), dict(w=P + 1), dict(rstd=P + 2), dict(o8=P, sc=None, group=64), dict(sc=P),
                dict(o8=P, sc=P, group=0), dict(o8=P, sc=P, group=-32), dict(o8=P, sc=P + 2, group=64),
                dict(o8=P, sc=P, group=64, ld8=255), dict(ro=P + 4096, ldro=264), dict(ro=P, ldro=264),
                dict(ro=P, kind=1), dict(out=P, ldo=264), dict(out=P + 8192), dict(out=P + 4096)):
        assert norm(**bad) == ARG, bad
    for bad in (dict(N=32769, ldx=40000, ldr=40000, ldro=40000, ldo=40000), dict(M=(1 << 24) + 1),
                dict(o8=P, sc=P, group=16), dict(o8=P, sc=P, group=96), dict(N=200, o8=P, sc=P, group=64)):
        assert norm(**bad) == UNS, bad


def test_norm_backward_validation():
    need = moe.moe_add_rms_norm_workspace_bytes(4, 64)

    def call(M=4, N=64, g=P, ldg=64, h=P + 4096, ldh=64, kind=0, r=P, w=P, d=P + 8192, ldd=64, dh=P + 16384, lddh=64,
             dw=P, ws=P, nbytes=need):
        return moe.lib().moe_add_rms_norm_backward(g, ldg, h, ldh, kind, r, M, N, w, d, ldd, dh, lddh, dw, ws, nbytes, None)

    assert call(M=0, g=None, h=None, r=None, dw=None, ws=None) == OK
    for bad in (dict(M=-1), dict(N=0), dict(kind=5), dict(g=None), dict(h=None), dict(r=None), dict(w=None),
                dict(dh=None, d=None, dw=None), dict(dh=None), dict(ldg=63), dict(ldh=60), dict(ldd=1), dict(lddh=63),
                dict(g=P + 1), dict(h=P + 2, kind=1), dict(dw=P + 2), dict(ws=None), dict(ws=P + 8), dict(r=P + 2),
                dict(M=0, ws=None), dict(dh=P + 8192, lddh=72), dict(dh=P + 4096, lddh=72), dict(dh=P, lddh=72),
                dict(dh=P, kind=1)):
        assert call(**bad) == ARG, bad
    assert call(nbytes=need - 1) == WS and call(N=40000, nbytes=1 << 40) == UNS
    assert call(M=(1 << 24) + 1, nbytes=1 << 40) == UNS
    assert moe.moe_add_rms_norm_workspace_bytes(-1, 8) == -1 and moe.moe_add_rms_norm_workspace_bytes(1, 0) == -1
    assert moe.moe_add_rms_norm_workspace_bytes(1, 32769) == -1


def test_workspaces_grow():
    for N in (1, 1000, 2048, 2049, 7168, 32768):
        sizes = [moe.moe_add_rms_norm_workspace_bytes(M, N) for M in [*range(3000), 1 << 20, 1 << 24]]
        assert sizes == sorted(sizes) and sizes[0] > 0
    sizes = [moe.moe_grad_norm_workspace_bytes(n) for n in range(8193)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    assert moe.moe_grad_norm_workspace_bytes(-1) == -1 and moe.moe_grad_norm_workspace_bytes(8193) == -1


def arrays(ptrs, sizes, kinds):
    n = len(ptrs)
    return (ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*sizes), (ctypes.c_int32 * n)(*kinds)


def test_grad_sumsq_validation():
    def call(ptrs=(P, P), sizes=(4, 4), kinds=(0, 1), n=2, out=P, ws=P, nbytes=1 << 30):
        a, s, k = arrays(ptrs, sizes, kinds)
        return moe.lib().moe_grad_sumsq(a, s, k, n, out, ws, nbytes, None)

    for bad in (dict(n=-1), dict(ptrs=(None, P)), dict(sizes=(4, -1)), dict(kinds=(0, 2)), dict(out=None), dict(out=P + 4),
                dict(ws=None), dict(ws=P + 8), dict(ptrs=(P + 1, P)), dict(ptrs=(P, P + 2))):
        assert call(**bad) == ARG, bad
    assert call(sizes=(4, (1 << 40) + 1)) == UNS
    assert call(nbytes=moe.moe_grad_norm_workspace_bytes(2) - 1) == WS
    lib = moe.lib()
    assert lib.moe_grad_sumsq(None, None, None, 1, P, P, 1 << 30, None) == ARG
    assert lib.moe_grad_sumsq(None, None, None, 8193, P, P, 1 << 30, None) == ARG


def test_grad_clip_validation():
    def call(ptrs, outs, sizes, kinds=None, most=1.0, sumsq=P, norm=None):
        a, s, k = arrays(ptrs, sizes, kinds or [1] * len(ptrs))
        o = (ctypes.c_void_p * len(outs))(*outs)
        return moe.lib().moe_grad_clip(a, o, s, k, len(ptrs), sumsq, most, norm, None)

    a, c = P, P + 4096
    for most in (-1.0, float("nan")):
        assert call([a], [a], [4], most=most) == ARG
    assert call([a], [a], [4], sumsq=None) == ARG and call([a], [a], [4], sumsq=P + 4) == ARG
    assert call([a], [a], [4], norm=P + 2) == ARG and call([a], [None], [4]) == ARG and call([a], [a + 2], [4]) == ARG
    # overlaps: out with out, out with another's gradient, out with a part of its own gradient
    for ptrs, outs, sizes in (([a, c], [a, a], [4, 4]), ([a, a], [a, a], [4, 4]), ([a, c], [c, a], [4, 4]),
                              ([a, c], [a, c - 4], [1024, 4]), ([a], [a + 4], [4]), ([a + 4], [a], [4]),
                              ([a, c, a + 8], [P + 65536, P + 131072, a], [8, 8, 2]),
                              ([a, c], [a, c - 1024], [1024, 1024])):
        assert call(ptrs, outs, sizes) == ARG, (ptrs, outs)


def test_clip_grad_norm_validation():
    def call(ptrs=(P,), outs=(P,), sizes=(4,), most=1.0, sumsq=P, norm=P, ws=P, nbytes=1 << 30):
        a, s, k = arrays(ptrs, sizes, [1] * len(ptrs))
        return moe.lib().moe_clip_grad_norm(a, (ctypes.c_void_p * len(outs))(*outs), s, k, len(ptrs), most, sumsq, norm, ws,
                                            nbytes, None)

    for bad in (dict(most=-1.0), dict(most=float("nan")), dict(sumsq=P + 4), dict(ws=None), dict(ws=P + 8), dict(norm=P + 2),
                dict(outs=(P + 4,)), dict(outs=(None,)), dict(ptrs=(None,)), dict(sizes=(-1,)),
                dict(ptrs=(P, P), outs=(P, P), sizes=(4, 4))):
        assert call(**bad) == ARG, bad
    assert call(nbytes=moe.moe_grad_norm_workspace_bytes(1) - 1) == WS


@pytest.fixture(scope="module")
def checker():
    import torch
    if torch.cuda.device_count() > 0:
        pytest.skip("host-only check: its calls pass host pointers, so it runs where no GPU is visible")
    if not os.path.exists(CLANG):
        pytest.skip("ROCm clang not found")
    folder = os.path.join(b.BUILD, "san_model")
    os.makedirs(folder, exist_ok=True)
    objs = []
    for src in b.sources():
        obj = os.path.join(b.BUILD, os.path.basename(src)[:-4] + ".o")
        if os.path.basename(src) == "abi_operators.hip":  # the entry points and their checks
            obj = os.path.join(folder, os.path.basename(src)[:-4] + ".o")
            _run([b.hipcc(), *b.COMMON, "-O1", "-g", "-fno-omit-frame-pointer", *SANITIZE_HOST, "-c", src, "-o", obj])
        elif not os.path.exists(obj) or os.path.getmtime(obj) < os.path.getmtime(src):
            os.makedirs(b.BUILD, exist_ok=True)
            obj = b._compile(src)
        objs.append(obj)
    drv = os.path.join(folder, "model_operator_checks.o")
    _run([CLANG, "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
          "-fno-sanitize-recover=all", "-I", os.path.join(b.ROOT, "include"), "-c",
          os.path.join(os.path.dirname(__file__), "model_operator_checks.c"), "-o", drv])
    exe = os.path.join(folder, "model_operator_checks")
    _run([CLANG + "++", "-fsanitize=address,undefined", drv, *objs, "-L/opt/rocm/lib", "-lamdhip64",
          "-Wl,-rpath,/opt/rocm/lib", "-o", exe])
    yield exe
    shutil.rmtree(folder, ignore_errors=True)


def test_model_operators_under_sanitizers(checker):
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:exitcode=23",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1:exitcode=24", HIP_VISIBLE_DEVICES="-1")
    r = subprocess.run([checker], capture_output=True, text=True, env=env, timeout=120)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out
    assert "runtime error" not in out and "AddressSanitizer" not in out, out
    assert "model operator checks passed" in r.stdout
