"""Refusals of the operators around the routed block (CPU only: every check
runs before any device work, and the pointers below are never followed)."""
import ctypes

import pytest
import torch

import nvfp4_moe_expert_topk_b200 as pkg

F = 1 << 40          # a 16-byte aligned address that nothing reads
P = ctypes.c_void_p
OK_BUT_NO_DEVICE = (-5, -6)


@pytest.fixture(scope="module")
def L():
    from nvfp4_moe_expert_topk_b200 import build
    build.build()
    return pkg.lib()


def norm_args(**kw):
    a = pkg.NormArgs()
    base = dict(x=F, residual=F, weight=F, T=4, H=256, ldx=256, ldr=256, ldro=256, ldy=256, eps=1e-6, residual_out=F,
                y=F, quant=1, scale_layout=0, gs=F, codes=F, scales=F)
    base.update(kw)
    for name, v in base.items():
        setattr(a, name, v)
    return a


def no_device():
    return not torch.cuda.is_available()


@pytest.mark.parametrize("change,status", [
    (dict(x=None), -1), (dict(weight=None), -1), (dict(T=-1), -1), (dict(H=0), -1), (dict(eps=-1.0), -1),
    (dict(eps=float("nan")), -1), (dict(quant=3), -1), (dict(scale_layout=2), -1), (dict(gs=None), -1),
    (dict(codes=None), -1), (dict(scales=None), -1), (dict(residual=None), -1), (dict(residual_out=None), -1),
    (dict(quant=0, y=None), -1), (dict(ldx=240), -1), (dict(ldr=0), -1), (dict(ldro=128), -1), (dict(ldy=255), -1),
    (dict(H=250), -2), (dict(H=32784, ldx=32784, ldr=32784, ldro=32784, ldy=32784), -2), (dict(T=1 << 31), -2),
    (dict(H=208, scale_layout=1), -2),
    (dict(x=F + 8), -3), (dict(residual=F + 2), -3), (dict(residual_out=F + 4), -3), (dict(weight=F + 2), -3),
    (dict(y=F + 8), -3), (dict(codes=F + 1), -3), (dict(scales=F + 1), -3), (dict(ldx=260), -3), (dict(ldr=257), -3),
    (dict(ldro=258), -3), (dict(ldy=264 + 4), -3),
])
def test_add_rmsnorm_refusals(L, change, status):
    assert L.nvfp4_add_rmsnorm(norm_args(**change), None) == status


def test_add_rmsnorm_accepts(L):
    """Forms that the checks have to let through (without a GPU the call then
    stops at the device check)."""
    assert L.nvfp4_add_rmsnorm(None, None) == -1
    if not no_device():
        pytest.skip("the pointers of this test are not real")
    for change in [dict(), dict(y=None), dict(quant=0, gs=None, codes=None, scales=None),
                   dict(quant=2, gs=None, H=208, scale_layout=7), dict(residual=None, residual_out=None),
                   dict(scale_layout=1), dict(T=0, x=None, weight=None, y=None, codes=None, scales=None, gs=None)]:
        assert L.nvfp4_add_rmsnorm(norm_args(**change), None) in OK_BUT_NO_DEVICE, change


def gemv(L, **kw):
    a = dict(x=F, M=4, ldx=256, codes=F, scales=F, gs=F, seg=(128, 200), nseg=None, N=200, K=256, out=F, ldo=200)
    a.update(kw)
    seg = None if a["seg"] is None else (ctypes.c_int64 * len(a["seg"]))(*a["seg"])
    nseg = a["nseg"] if a["nseg"] is not None else len(a["seg"] or ())
    return L.nvfp4_gemv(a["x"], a["M"], a["ldx"], a["codes"], a["scales"], a["gs"], seg, nseg, a["N"], a["K"],
                        a["out"], a["ldo"], None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), -1), (dict(out=None), -1), (dict(codes=None), -1), (dict(scales=None), -1), (dict(gs=None), -1),
    (dict(seg=None, nseg=1), -1), (dict(nseg=0), -1), (dict(M=-1), -1), (dict(N=0, seg=(1,)), -1), (dict(K=0), -1),
    (dict(ldx=128), -1), (dict(ldo=199), -1), (dict(seg=(128, 199)), -1), (dict(seg=(200, 200)), -1),
    (dict(seg=(0, 200)), -1), (dict(seg=(220, 200)), -1),
    (dict(M=17), -2), (dict(K=224), -2), (dict(K=(1 << 20) + 64, ldx=(1 << 20) + 64), -2),
    (dict(N=1 << 31, seg=(1 << 31,), ldo=1 << 31), -2), (dict(seg=(1, 2, 3, 4, 200)), -2),
    (dict(x=F + 8), -3), (dict(codes=F + 8), -3), (dict(scales=F + 4), -3), (dict(gs=F + 2), -3), (dict(out=F + 1), -3),
    (dict(ldx=260), -3),
])
def test_gemv_refusals(L, change, status):
    assert gemv(L, **change) == status


def test_gemv_accepts(L):
    if not no_device():
        pytest.skip("the pointers of this test are not real")
    for change in [dict(), dict(M=0, x=None, out=None), dict(M=16), dict(seg=(7, 31, 199, 200)), dict(ldo=1001),
                   dict(out=F + 2)]:
        assert gemv(L, **change) in OK_BUT_NO_DEVICE, change


def balance(L, **kw):
    a = dict(logits=F, ids=F, ld=6, T=100, E=48, k=6, off=F, S=3, scoring=0, counts=F, tokens=F, probs=F, loss=F, ws=F,
             nbytes=1 << 30)
    a.update(kw)
    return L.nvfp4_moe_balance(a["logits"], a["ids"], a["ld"], a["T"], a["E"], a["k"], a["off"], a["S"], a["scoring"],
                               a["counts"], a["tokens"], a["probs"], a["loss"], a["ws"], a["nbytes"], None)


def backward(L, **kw):
    a = dict(logits=F, ids=F, ld=6, T=100, E=48, k=6, off=F, S=3, scoring=0, counts=F, tokens=F, gl=F, gw=F, out=F)
    a.update(kw)
    return L.nvfp4_moe_balance_backward(a["logits"], a["ids"], a["ld"], a["T"], a["E"], a["k"], a["off"], a["S"],
                                        a["scoring"], a["counts"], a["tokens"], a["gl"], a["gw"], a["out"], None)


SHARED = [
    (dict(logits=None), -1), (dict(ids=None), -1), (dict(T=-1), -1), (dict(E=0), -1), (dict(k=0), -1), (dict(ld=5), -1),
    (dict(S=0), -1), (dict(scoring=2), -1), (dict(off=None), -1), (dict(counts=None), -1), (dict(tokens=None), -1),
    (dict(E=1025), -2), (dict(k=33, ld=33), -2), (dict(E=4), -2), (dict(T=1 << 31), -2), (dict(S=65536), -2),
]


@pytest.mark.parametrize("change,status", SHARED + [
    (dict(probs=None), -1), (dict(loss=None), -1), (dict(ws=None), -1), (dict(ws=F + 8), -3), (dict(nbytes=100), -4)])
def test_balance_refusals(L, change, status):
    assert balance(L, **change) == status


@pytest.mark.parametrize("change,status", SHARED + [(dict(gl=None), -1), (dict(out=None), -1)])
def test_balance_backward_refusals(L, change, status):
    assert backward(L, **change) == status


def test_balance_accepts(L):
    if not no_device():
        pytest.skip("the pointers of this test are not real")
    for change in [dict(), dict(off=None, S=1), dict(T=0, logits=None, ids=None), dict(ld=7),
                   dict(nbytes=L.nvfp4_moe_balance_workspace_size(100, 3, 48))]:
        assert balance(L, **change) in OK_BUT_NO_DEVICE, change
    for change in [dict(), dict(gw=None), dict(T=0, logits=None, ids=None, out=None)]:
        assert backward(L, **change) in OK_BUT_NO_DEVICE, change


def test_balance_workspace_size(L):
    n = L.nvfp4_moe_balance_workspace_size
    assert n(-1, 1, 8) == 0 and n(10, 0, 8) == 0 and n(10, 1, 1025) == 0
    assert n(0, 1, 1) > 0
    last = 0
    for T in (1, 100, 5000, 100000, 1 << 24):       # grows with the batch, and stays small beside its logits
        now = n(T, 4, 384)
        assert now >= last
        last = now
    assert last < (1 << 24) * 384 * 4 // 100


def test_binding_refusals(L):
    """What the binding itself refuses, before the library is called."""
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    w = torch.zeros(256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        pkg.nvfp4_add_rmsnorm(x, w, 1e-6, y=x)
    with pytest.raises(ValueError, match="x is required"):
        pkg.nvfp4_add_rmsnorm(None, w, 1e-6, y=x)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        pkg.nvfp4_gemv(x, x, x, x, [4], x)
    with pytest.raises(ValueError, match="logits must be a CUDA tensor"):
        pkg.nvfp4_moe_balance(torch.zeros(4, 8), None, 2, None, None, None, None, None)
    with pytest.raises(ValueError, match="logits is required"):
        pkg.nvfp4_moe_balance_backward(None, None, 2, None, None, None, None)


def test_binding_argument_kinds(L):
    """Arguments of another kind end in a Python error, and a refused call
    keeps no reference to what it was given."""
    import sys

    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    for wrong in (3, [x], "x", object()):
        with pytest.raises(ValueError, match="x must be a CUDA tensor"):
            pkg.nvfp4_add_rmsnorm(wrong, x, 1e-6, y=x)
        with pytest.raises(ValueError, match="logits must be a CUDA tensor"):
            pkg.nvfp4_moe_balance(wrong, x, 2, x, x, x, x, x)
    native = pkg._binding()
    for name, n in (("add_rmsnorm", 12), ("gemv", 7), ("balance", 11), ("backward", 11)):
        for got in (0, n - 1, n + 1):
            with pytest.raises(ValueError, match=f"expected {n} arguments, got {got}"):
                getattr(native, name)(*[x] * got)
    before = sys.getrefcount(x)
    for _ in range(50):
        with pytest.raises(ValueError):
            pkg.nvfp4_add_rmsnorm(x, x, 1e-6, y=x, residual=x, residual_out=x, codes=x, scales=x, gs=x)
    assert sys.getrefcount(x) == before


@pytest.mark.parametrize("S", [1, 2, 4, 33, 147, 148, 149, 1000])
@pytest.mark.parametrize("E", [1, 48, 384, 512, 513, 1024])
def test_balance_workspace_of_a_long_batch_serves_shorter_ones(L, E, S):
    """A caller sizes its workspace once, for its largest batch: the size does
    not shrink as T, S or E grow (every T over the borders between chunk lengths)."""
    n = L.nvfp4_moe_balance_workspace_size
    last = 0
    around = [128 * w * S + d for w in (12, 16) for d in (-1, 0, 1)]
    for T in sorted(set(range(6000)) | set(range(6000, 300000, 997)) | set(around)):
        assert n(T, S, E) >= last, T
        last = n(T, S, E)
    for T in (1, 700, 2000, 128 * 12 * S, 128 * 16 * S, 128 * 16 * S + 1, 100000):
        assert n(T, S, E) <= n(T, S + 1, E) and n(T, S, E) <= n(T + 1, S, E)
        if E < 1024:
            assert n(T, S, E) <= n(T, S, E + 1)


def test_balance_takes_a_workspace_of_a_longer_batch(L):
    if not no_device():
        pytest.skip("the pointers of this test are not real")
    size = max(L.nvfp4_moe_balance_workspace_size(3000, 1, 384), L.nvfp4_moe_balance_workspace_size(2049, 1, 384))
    for T in (1, 100, 1999, 2000, 2047, 2048, 2049, 3000):
        assert balance(L, T=T, E=384, off=None, S=1, nbytes=size) in OK_BUT_NO_DEVICE, T
