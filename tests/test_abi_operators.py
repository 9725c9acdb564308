"""Host-side checks of the operators' entry points (no GPU): sizes, statuses
before any launch, and the same calls with extreme sizes in a build of the
host code with AddressSanitizer and UndefinedBehaviorSanitizer."""
import os
import shutil
import subprocess

import pytest

import int4_weight_only_moe_amd as moe
from int4_weight_only_moe_amd import build as b
from test_abi_sanitize import CLANG, SANITIZE_HOST, _run

P = 0x10000  # an aligned non-null address; validation fails before any use
ARG, UNS, WS = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE


def balance(M=4, E=384, k=8, off=P, S=2, ptr=P, logits=P, ws=P, nbytes=None):
    if nbytes is None:
        nbytes = moe.moe_balance_workspace_bytes(max(M, 0), E, max(S, 1))
    return moe.lib().moe_balance_loss(logits, P, M, E, k, off, S, None, ptr, ptr, ptr, ptr, ws, nbytes, None)


def test_balance_validation():
    assert balance(M=-1) == ARG and balance(E=0) == ARG and balance(k=0) == ARG and balance(S=0) == ARG
    assert balance(off=None) == ARG  # more than one sequence needs offsets
    assert balance(E=1025, nbytes=1 << 30) == UNS
    assert balance(k=17) == UNS and balance(E=4, k=5) == UNS and balance(S=65536, nbytes=1 << 30) == UNS
    assert balance(M=1 << 27, nbytes=1 << 40) == UNS  # M * top_k >= 2^30
    assert balance(logits=None) == ARG and balance(ptr=None) == ARG and balance(ws=None) == ARG
    assert balance(logits=P + 2) == ARG and balance(ptr=P + 1) == ARG and balance(ws=P + 8) == ARG
    assert balance(off=P + 2) == ARG
    assert balance(M=0, logits=None, ptr=None) == ARG  # the outputs of an empty batch are written
    assert balance(nbytes=moe.moe_balance_workspace_bytes(4, 384, 2) - 1) == WS
    assert moe.moe_balance_workspace_bytes(-1, 8, 1) == -1 and moe.moe_balance_workspace_bytes(1, 1025, 1) == -1
    assert moe.moe_balance_workspace_bytes(1, 8, 0) == -1


def test_balance_backward_validation():
    def call(M=4, E=8, k=2, off=None, S=1, logits=P, p=P, grad=P):
        return moe.lib().moe_balance_loss_backward(logits, M, E, k, off, S, None, p, p, p, grad, None)

    assert call(M=0, logits=None, p=None, grad=None) == moe.MOE_OK
    assert call(M=-1) == ARG and call(S=2) == ARG and call(logits=None) == ARG and call(p=None) == ARG
    assert call(grad=None) == ARG and call(grad=P + 2) == ARG and call(E=2048, k=2) == UNS and call(k=9) == UNS


def forward(M=4, L=2, K=64, N=48, r=16, x=P, ldx=64, base=P, ldb=48, out=P, ldo=48, kind=0, h=None, a=P, ids=P,
            scales=None, nbytes=1 << 50, ws=P):
    return moe.lib().moe_lora_forward(x, ldx, ids, M, L, K, N, r, a, P, scales, base, ldb, out, ldo, kind, h, ws,
                                      nbytes, None)


def test_lora_forward_validation():
    assert forward(M=0, x=None, ids=None, base=None, out=None, ws=None) == moe.MOE_OK
    for bad in (dict(M=-1), dict(L=0), dict(K=0), dict(N=0), dict(r=0), dict(kind=2), dict(x=None), dict(ids=None),
                dict(a=None), dict(out=None), dict(ws=None), dict(x=P + 8), dict(a=P + 8), dict(ldx=56), dict(ldx=68),
                dict(ldb=47), dict(ldo=40), dict(ldb=56), dict(out=P + 1), dict(base=P + 2, kind=1),
                dict(h=P + 8), dict(scales=P + 2), dict(ws=P + 4), dict(ids=P + 1)):
        assert forward(**bad) == ARG, bad
    for bad in (dict(L=1025), dict(r=12), dict(r=136), dict(K=60), dict(M=(1 << 24) + 1), dict(K=(1 << 20) + 8),
                dict(N=(1 << 20) + 1)):
        assert forward(**bad) == UNS, bad
    need = moe.moe_lora_workspace_bytes(4, 2, 64, 48, 16, False)
    assert forward(nbytes=need - 1) == WS


def test_lora_backward_validation():
    def call(M=4, L=2, K=64, N=48, r=16, g=P, ldg=48, kind=0, x=P, ldx=64, ids=P, h=P, dxb=P, ldxb=64, dx=P, ldd=64,
             ga=P, gb=P, ws=P, nbytes=1 << 50):
        return moe.lib().moe_lora_backward(g, ldg, kind, x, ldx, ids, h, M, L, K, N, r, P, P, None, dxb, ldxb, dx, ldd,
                                           ga, gb, ws, nbytes, None)

    for bad in (dict(M=-1), dict(kind=-1), dict(g=None), dict(x=None), dict(h=None), dict(ids=None), dict(dx=None),
                dict(ga=None), dict(gb=None), dict(ws=None), dict(ldg=40), dict(ldx=60), dict(ldd=70), dict(ldxb=72),
                dict(ga=P + 4), dict(h=P + 4), dict(dx=P + 8), dict(g=P + 1), dict(M=0, ga=None)):
        assert call(**bad) == ARG, bad
    assert call(r=20) == UNS and call(L=5000) == UNS
    assert call(nbytes=moe.moe_lora_workspace_bytes(4, 2, 64, 48, 16, True) - 1) == WS
    assert moe.moe_lora_workspace_bytes(4, 2, 64, 48, 12, True) == -1
    assert moe.moe_lora_workspace_bytes(0, 2, 64, 48, 8, True) > 0


def test_workspaces_grow_with_the_batch():
    """A workspace for more rows serves fewer, and a backward call's the forward call."""
    for L, K, N, r in ((1, 7168, 7168, 64), (1024, 64, 1, 8), (8, 8, 5000, 128), (64, 2048, 384, 24)):
        before = {0: 0, 1: 0}
        for M in [*range(0, 300), *range(300, 20000, 97), 100000, 1 << 22, 1 << 24]:
            need = {back: moe.moe_lora_workspace_bytes(M, L, K, N, r, back) for back in (0, 1)}
            assert need[1] >= need[0] and need[0] >= before[0] and need[1] >= before[1], M
            before = need
    for E in (1, 384, 1024):
        sizes = [moe.moe_balance_workspace_bytes(M, E, 5) for M in [*range(0, 3000, 7), *range(3000, 100000, 613)]]
        assert sizes == sorted(sizes)


@pytest.fixture(scope="module")
def checker():
    import torch
    if torch.cuda.device_count() > 0:
        pytest.skip("host-only check: its calls pass host pointers, so it runs where no GPU is visible")
    if not os.path.exists(CLANG):
        pytest.skip("ROCm clang not found")
    folder = os.path.join(b.BUILD, "san_operators")
    os.makedirs(folder, exist_ok=True)
    objs = []
    for src in b.sources():
        obj = os.path.join(b.BUILD, os.path.basename(src)[:-4] + ".o")
        if os.path.basename(src) in ("abi_operators.hip", "balance.hip", "lora.hip"):
            # the entry points, and the files that hold their layouts' sizes
            obj = os.path.join(folder, os.path.basename(src)[:-4] + ".o")
            _run([b.hipcc(), *b.COMMON, "-O1", "-g", "-fno-omit-frame-pointer", *SANITIZE_HOST, "-c", src, "-o", obj])
        elif not os.path.exists(obj) or os.path.getmtime(obj) < os.path.getmtime(src):
            os.makedirs(b.BUILD, exist_ok=True)
            obj = b._compile(src)
        objs.append(obj)
    drv = os.path.join(folder, "operator_checks.o")
    _run([CLANG, "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
          "-fno-sanitize-recover=all", "-I", os.path.join(b.ROOT, "include"), "-c",
          os.path.join(os.path.dirname(__file__), "operator_checks.c"), "-o", drv])
    exe = os.path.join(folder, "operator_checks")
    _run([CLANG + "++", "-fsanitize=address,undefined", drv, *objs, "-L/opt/rocm/lib", "-lamdhip64",
          "-Wl,-rpath,/opt/rocm/lib", "-o", exe])
    yield exe
    shutil.rmtree(folder, ignore_errors=True)


def test_operators_validation_under_sanitizers(checker):
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:exitcode=23",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1:exitcode=24", HIP_VISIBLE_DEVICES="-1")
    r = subprocess.run([checker], capture_output=True, text=True, env=env, timeout=120)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out
    assert "runtime error" not in out and "AddressSanitizer" not in out, out
    assert "operator checks passed" in r.stdout
