"""The operators around the routed block as programs use them beyond one call
at a time: first call inside a capture, several streams at once, another
current device, positions past 32 bits."""
import subprocess
import sys

import pytest
import torch

import nvfp4_moe_expert_topk_b200 as lib
from conftest import ROOT

pytestmark = pytest.mark.gpu
DEV = "cuda"


def bits(t):
    return t.view(torch.int16)


def norm_call(T, H, seed, quant=lib.NVFP4_QUANT_NVFP4):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    r = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    w = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    gs = torch.tensor([400.0], device=DEV)
    out = [torch.empty_like(x), torch.empty_like(x), torch.empty(T, H // 2, dtype=torch.uint8, device=DEV),
           torch.empty(T, H // 16, dtype=torch.uint8, device=DEV)]
    return out, lambda s=None: lib.nvfp4_add_rmsnorm(x, w, 1e-6, y=out[0], residual=r, residual_out=out[1], quant=quant,
                                                     gs=gs, codes=out[2], scales=out[3], stream=s)


def gemv_call(M, N, K, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(M, K, generator=g, device=DEV).to(torch.bfloat16)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.randint(8, 120, ((N + 127) // 128 * 128 * (K // 16),), generator=g, device=DEV, dtype=torch.uint8)
    gs = torch.tensor([3.0], device=DEV)
    out = [torch.empty(M, N, dtype=torch.bfloat16, device=DEV)]
    return out, lambda s=None: lib.nvfp4_gemv(x, codes, scales, gs, [N], out[0], stream=s)


def balance_call(T, E, k, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    l = torch.randn(T, E, generator=g, device=DEV)
    ids = torch.topk(l, k).indices.to(torch.int32)
    off = torch.tensor([0, T // 3, T // 2, T], dtype=torch.int32, device=DEV)
    out = [torch.empty(3, E, dtype=torch.int32, device=DEV), torch.empty(3, dtype=torch.int32, device=DEV),
           torch.empty(3, E, device=DEV), torch.empty(3, device=DEV), torch.empty(T, E, device=DEV)]
    ws = torch.empty(lib.nvfp4_moe_balance_workspace_size(T, 3, E), dtype=torch.uint8, device=DEV)
    gw = torch.randn(T, k, generator=g, device=DEV)
    gl = torch.ones(3, device=DEV)

    def call(s=None):
        lib.nvfp4_moe_balance(l, ids, k, *out[:4], ws, seq_offsets=off, stream=s)
        lib.nvfp4_moe_balance_backward(l, ids, k, out[0], out[1], gl, out[4], gw, seq_offsets=off, stream=s)
    return out, call


CALLS = [(norm_call, (300, 1536)), (norm_call, (1, 7168)), (gemv_call, (3, 640, 4096)), (gemv_call, (16, 4096, 512)),
         (gemv_call, (1, 64, 8192)), (balance_call, (100, 48, 6)), (balance_call, (5000, 384, 6))]


@pytest.mark.parametrize("make,args", CALLS)
def test_streams_at_once(make, args):
    """The same operator on four streams at a time, each with its own data,
    gives what it gives alone."""
    calls = [make(*args, seed) for seed in range(4)]
    alone = []
    for out, call in calls:
        call()
        torch.cuda.synchronize()
        alone.append([t.clone() for t in out])
        for t in out:
            t.zero_()
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        for (out, call), s in zip(calls, streams):
            call(s)
    torch.cuda.synchronize()
    for (out, _), want in zip(calls, alone):
        for a, b in zip(out, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("make,args", CALLS)
def test_calls_back_to_back(make, args):
    """Consecutive calls on one stream, without a wait between them, each
    reading what the one before wrote."""
    out, call = make(*args, 7)
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in out]
    for _ in range(30):
        for t in out:
            t.zero_()
        call()
    torch.cuda.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a, b)


FIRST = """
import sys, torch
sys.path[:0] = [{root!r}, {tests!r}]
import test_gpu_layer_use as t
out, call = t.{make}(*{args!r}, 3)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    call()
for o in out:
    o.zero_()
graph.replay()
torch.cuda.synchronize()
got = [o.clone() for o in out]
call()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, out)), "replay differs"
print("same")
"""


@pytest.mark.parametrize("make,args", [("norm_call", (40, 1536)), ("gemv_call", (5, 512, 4096)), ("gemv_call", (16, 4096, 512)),
                                       ("balance_call", (5000, 384, 6)), ("balance_call", (90, 1024, 6))])
def test_first_call_may_be_captured(make, args):
    """A process's first call of an operator inside a stream capture."""
    code = FIRST.format(root=ROOT, tests=ROOT + "/tests", make=make, args=args)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two devices")
@pytest.mark.parametrize("make,args", CALLS)
def test_other_current_device(make, args):
    out, call = make(*args, 1)
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in out]
    for t in out:
        t.zero_()
    torch.cuda.synchronize()
    with torch.cuda.device(1):
        call()
    torch.cuda.synchronize(0)
    for a, b in zip(out, want):
        assert torch.equal(a, b)


# ---- positions past 2^31 elements or bytes: the last rows equal a small call's on a copy of them
def test_norm_past_32_bits():
    T, H = 300000, 7168                                  # 2.15e9 elements
    x = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    x[-64:] = torch.randn(64, H, device=DEV).to(torch.bfloat16)
    x[:-64] = 1.0
    w = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    codes = torch.empty(T, H, dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.empty(T, H // 128, device=DEV)
    y = torch.empty_like(x)
    lib.nvfp4_add_rmsnorm(x, w, 1e-6, y=y, quant=lib.NVFP4_QUANT_E4M3, codes=codes, scales=scales)
    y2, c2, s2 = torch.empty(64, H, dtype=torch.bfloat16, device=DEV), torch.empty(64, H, dtype=torch.float8_e4m3fn, device=DEV), torch.empty(64, H // 128, device=DEV)
    lib.nvfp4_add_rmsnorm(x[-64:].clone(), w, 1e-6, y=y2, quant=lib.NVFP4_QUANT_E4M3, codes=c2, scales=s2)
    assert torch.equal(bits(y[-64:]), bits(y2)) and torch.equal(scales[-64:], s2)
    assert torch.equal(codes[-64:].view(torch.uint8), c2.view(torch.uint8))
    assert (bits(y[:1000]) == bits(y[:1, :1])).all()


def test_gemv_past_32_bits():
    N, K, M = 1 << 20, 8192, 2                           # 4.3e9 bytes of codes
    codes = torch.randint(0, 256, (N, K // 2), device=DEV, dtype=torch.uint8)
    scales = torch.randint(8, 120, (N * (K // 16),), device=DEV, dtype=torch.uint8)
    gs = torch.tensor([2.0], device=DEV)
    x = torch.randn(M, K, device=DEV).to(torch.bfloat16)
    out = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    lib.nvfp4_gemv(x, codes, scales, gs, [N], out)
    last = torch.empty(M, 256, dtype=torch.bfloat16, device=DEV)
    lib.nvfp4_gemv(x, codes[-256:].clone(), scales[-256 * (K // 16):].clone(), gs, [256], last)
    a, b = out[:, -256:].double(), last.double()
    # the two split k differently: each within (K / 8 + 33) 2^-23 of the sum of magnitudes and a bf16 rounding
    mag = x.double().abs().sum(dim=1, keepdim=True) * 6 * 2.0 ** 9 / 2.0
    assert ((a - b).abs() <= 2 * 2.0 ** -8 * b.abs() + 2 * (K / 8 + 33) * 2.0 ** -23 * mag).all()
    assert b.abs().max() > 0


def test_balance_past_32_bits():
    T, E, k = 2200000, 1024, 4                           # 2.25e9 logits
    n = 700
    l = torch.zeros(T, E, device=DEV)
    l[-n:] = torch.randn(n, E, device=DEV)
    ids = torch.zeros(T, k, dtype=torch.int32, device=DEV)
    ids[:] = torch.arange(k, dtype=torch.int32, device=DEV)
    ids[-n:] = torch.topk(l[-n:], k).indices.to(torch.int32)
    gw = torch.zeros(T, k, device=DEV)
    gw[-n:] = torch.randn(n, k, device=DEV)
    gl = torch.ones(2, device=DEV)

    def run(l, ids, gw, off, S):
        out = [torch.empty(S, E, dtype=torch.int32, device=DEV), torch.empty(S, dtype=torch.int32, device=DEV),
               torch.empty(S, E, device=DEV), torch.empty(S, device=DEV)]
        ws = torch.empty(lib.nvfp4_moe_balance_workspace_size(l.shape[0], S, E), dtype=torch.uint8, device=DEV)
        lib.nvfp4_moe_balance(l, ids, k, *out, ws, seq_offsets=off)
        grad = torch.empty_like(l)
        lib.nvfp4_moe_balance_backward(l, ids, k, out[0], out[1], gl[:S], grad, gw, seq_offsets=off)
        return out, grad
    (c, t, p, loss), grad = run(l, ids, gw, torch.tensor([0, T - n, T], dtype=torch.int32, device=DEV), 2)
    (c2, t2, p2, loss2), grad2 = run(l[-n:].clone(), ids[-n:].clone(), gw[-n:].clone(), None, 1)
    assert torch.equal(c[1], c2[0]) and int(t[1]) == n and int(t[0]) == T - n
    assert int(c[0, 0]) == T - n
    assert torch.allclose(p[1], p2[0], rtol=1e-5) and torch.allclose(loss[1], loss2[0], rtol=1e-5)
    assert torch.equal(grad[-n:], grad2)                 # a row's gradient does not depend on the batch around it


@pytest.mark.parametrize("make,args", CALLS)
def test_threads_at_once(make, args):
    """Four threads, each with its own data and stream (the interpreter lock
    is not held while a call launches)."""
    import threading

    calls = [make(*args, seed) for seed in range(4)]
    alone = []
    for out, call in calls:
        call()
        torch.cuda.synchronize()
        alone.append([t.clone() for t in out])
        for t in out:
            t.zero_()
    torch.cuda.synchronize()
    errors = []

    def work(call, stream):
        try:
            for _ in range(50):
                call(stream)
        except Exception as e:          # reported by the test's own thread
            errors.append(e)

    streams = [torch.cuda.Stream() for _ in calls]
    threads = [threading.Thread(target=work, args=(call, s)) for (_, call), s in zip(calls, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for (out, _), want in zip(calls, alone):
        for a, b in zip(out, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_current_stream_is_used():
    """Without a stream argument the call goes to the current stream."""
    out, call = norm_call(300, 1536, 9)
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in out]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):     # a launch on another stream would not be recorded
        call()
    for t in out:
        t.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_wrong_kinds_of_arguments():
    x = torch.zeros(2, 256, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(256, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(TypeError):
        lib.nvfp4_add_rmsnorm(x, w, "small", y=x)
    with pytest.raises(TypeError):
        lib.nvfp4_add_rmsnorm(x, w, 1e-6, y=x, quant="nvfp4")
    with pytest.raises(AttributeError):
        lib.nvfp4_add_rmsnorm(x, w, 1e-6, y=x, stream=7)
    with pytest.raises(ValueError, match="x must be .T, H., got .256."):
        lib.nvfp4_add_rmsnorm(w, w, 1e-6, y=x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        lib.nvfp4_add_rmsnorm(x, w, 1e-6, y=x.to_sparse())
    codes = torch.zeros(64, 128, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(128 * 16, dtype=torch.uint8, device=DEV)
    gs, out = torch.ones(1, device=DEV), torch.empty(2, 64, dtype=torch.bfloat16, device=DEV)
    for seg in (64, None, ["a"], [1.5]):
        with pytest.raises(TypeError):
            lib.nvfp4_gemv(x, codes, scales, gs, seg, out)
    with pytest.raises(lib.Nvfp4Error) as e:
        lib.nvfp4_gemv(x, codes, scales, torch.ones(5, device=DEV), [1, 2, 3, 4, 64], out)
    assert e.value.status == -2
    for seg in ((64,), torch.tensor([64])):
        lib.nvfp4_gemv(x, codes, scales, gs, seg, out)
    l = torch.zeros(8, 16, device=DEV)
    ids = torch.zeros(8, 2, dtype=torch.int32, device=DEV)
    c, t = torch.zeros(1, 16, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    p, s = torch.zeros(1, 16, device=DEV), torch.zeros(1, device=DEV)
    ws = torch.empty(lib.nvfp4_moe_balance_workspace_size(8, 1, 16), dtype=torch.uint8, device=DEV)
    for k in (None, "2", 2.0):
        with pytest.raises(TypeError):
            lib.nvfp4_moe_balance(l, ids, k, c, t, p, s, ws)
    with pytest.raises(ValueError, match="out of range"):
        lib.nvfp4_moe_balance(l, ids, 2, c, t, p, s, ws, scoring=1 << 40)
    for n in (0, 1):
        with pytest.raises(ValueError, match="seq_offsets must hold"):
            lib.nvfp4_moe_balance(l, ids, 2, c, t, p, s, ws, seq_offsets=t[:n])
    with pytest.raises(lib.Nvfp4Error) as e:
        lib.nvfp4_moe_balance(l, ids, 0, c, t, p, s, ws)
    assert e.value.status == -1
    lib.nvfp4_moe_balance(l, ids, 2, c, t, p, s, ws)


def in_new_thread(call):
    import threading

    errors = []

    def work():
        try:
            call()
        except Exception as e:
            errors.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not errors, errors


@pytest.mark.parametrize("make,args", CALLS)
def test_first_call_of_a_thread(make, args):
    out, call = make(*args, 3)
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in out]
    for t in out:
        t.zero_()
    in_new_thread(call)
    for a, b in zip(out, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_first_call_of_a_thread_dense_gemm():
    """The dense product builds tensor maps before its first launch, like the
    few-row one."""
    M, N, K = 130, 256, 512
    g = torch.Generator(device=DEV).manual_seed(1)

    def operand(rows):
        codes = torch.randint(0, 256, (rows, K // 2), generator=g, device=DEV, dtype=torch.uint8)
        scales = torch.randint(8, 100, (lib.nvfp4_scales_bytes(rows, K, lib.NVFP4_SCALES_MMA),), generator=g, device=DEV,
                               dtype=torch.uint8)
        return codes, scales, torch.ones(1, device=DEV)

    a, b = operand(M), operand(N)
    want, out = (torch.zeros(M, N, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    lib.nvfp4_gemm(*a, *b, [N], want)
    in_new_thread(lambda: lib.nvfp4_gemm(*a, *b, [N], out))
    assert want.abs().sum() > 0 and torch.equal(bits(out), bits(want))
