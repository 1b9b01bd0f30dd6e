"""nvfp4_add_rmsnorm against its definition.

Everything is compared bit for bit.  h is one rounding of an exact sum; the
sum of squares is held in 64 bits on both sides and its orders of summation
differ by ~1e-16 relative, so the fp32 rstd is the same unless it lies within
that of a rounding border (about one row in 10^8); the products, the bf16
rounding and the quantisation are single IEEE steps on equal operands.  The
NVFP4 rows are the oracle quantiser's on the bf16 row."""
import numpy as np
import pytest
import torch

import oracle as O
from helpers import from_mma_layout
from nvfp4_moe_expert_topk_b200 import (NVFP4_QUANT_E4M3, NVFP4_QUANT_NONE, NVFP4_QUANT_NVFP4, NVFP4_SCALES_MMA,
                                        NVFP4_SCALES_ROWMAJOR, nvfp4_add_rmsnorm, nvfp4_scales_bytes)
from nvfp4_moe_expert_topk_b200 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6


def rows(T, H, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g) * torch.exp(torch.empty(T, 1).uniform_(-spread, spread, generator=g))
    loud = torch.rand(H, generator=g) < 0.02
    x[:, loud] *= 20
    return x.to(torch.bfloat16)


def reference(x, res, w, eps=EPS):
    """(h bf16, y fp32) on the CPU."""
    h = x if res is None else (x.double() + res.double()).to(torch.bfloat16)
    hd = h.double().numpy()
    rstd = (1.0 / np.sqrt((hd * hd).sum(axis=1, keepdims=True) / h.shape[1] + eps)).astype(np.float32)
    y = (h.float().numpy() * rstd) * w.float().numpy()
    assert y.dtype == np.float32
    return h, y


def bits(t):
    return t.cpu().contiguous().view(torch.int16)


def e4m3_rows(y):
    """(code bytes, scales) of fp32 rows, groups of 128 columns."""
    T, H = y.shape
    G = (H + 127) // 128
    pad = np.zeros((T, G * 128), np.float32)
    pad[:, :H] = y
    grp = pad.reshape(T, G, 128)
    a = np.abs(grp).max(axis=2)
    with np.errstate(divide="ignore"):
        r = np.where(a == 0, np.float32(0), np.float32(448.0) / a).astype(np.float32)
    q = torch.from_numpy((grp * r[:, :, None]).reshape(T, -1)[:, :H].copy()).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8), a / np.float32(448.0)


def check(T, H, quant, layout=NVFP4_SCALES_ROWMAJOR, res=True, y=True, pads=(0, 0, 0, 0), seed=0, x=None, r=None,
          gs_value=60.0):
    """One call with row strides H + pads, surrounded by guard values."""
    x = rows(T, H, 10 * seed + 1) if x is None else x
    r = (rows(T, H, 10 * seed + 2) if r is None else r) if res else None
    w = (1 + 0.2 * torch.randn(H, generator=torch.Generator().manual_seed(seed))).to(torch.bfloat16)
    want_h, want_y = reference(x, r, w)

    def strided(src, pad):
        buf = torch.full((T, H + pad), 77.0, dtype=torch.bfloat16, device=DEV)
        if src is not None:
            buf[:, :H] = src.to(DEV)
        return buf
    xb, rb, ob, yb = strided(x, pads[0]), strided(r, pads[1]), strided(None, pads[2]), strided(None, pads[3])
    gs = torch.tensor([gs_value], device=DEV)
    codes = scales = None
    if quant == NVFP4_QUANT_NVFP4:
        codes = torch.full((T + 1, H // 2), 0xA5, dtype=torch.uint8, device=DEV)
        n = nvfp4_scales_bytes(T, H, layout)
        scales = torch.full((n + 16,), 0xA5, dtype=torch.uint8, device=DEV)
    elif quant == NVFP4_QUANT_E4M3:
        codes = torch.full((T + 1, H), 0xA5, dtype=torch.uint8, device=DEV)
        scales = torch.full((T + 1, (H + 127) // 128), -3.0, device=DEV)
    cv = None if codes is None else codes[:T]
    sv = None if scales is None else (scales[:n] if quant == NVFP4_QUANT_NVFP4 else scales[:T])
    nvfp4_add_rmsnorm(xb[:, :H], w.to(DEV), EPS, y=yb[:, :H] if y else None, residual=rb[:, :H] if res else None,
                      residual_out=ob[:, :H] if res else None, quant=quant, gs=gs, codes=cv, scales=sv,
                      scale_layout=layout)
    torch.cuda.synchronize()
    want_b = torch.from_numpy(want_y).to(torch.bfloat16)
    if res:
        assert torch.equal(bits(ob[:, :H]), bits(want_h))
    if y:
        assert torch.equal(bits(yb[:, :H]), bits(want_b))
    for buf in (xb, rb, ob, yb):                       # nothing outside the windows
        assert (buf[:, H:] == 77.0).all()
    if not y:
        assert (yb == 77.0).all()
    if quant == NVFP4_QUANT_NVFP4:
        wc, wsc = O.quantize_bf16(W.bf16_bits(want_b), np.float32(gs_value))
        assert np.array_equal(codes[:T].cpu().numpy(), wc)
        assert (codes[T] == 0xA5).all() and (scales[n:] == 0xA5).all()
        got = scales[:n].cpu().numpy()
        if layout == NVFP4_SCALES_MMA:
            assert np.array_equal(from_mma_layout(got, T, H), wsc)
            full = np.full(((T + 127) // 128 * 128, H // 16), 0, np.uint8)
            full[:T] = 1                                # pad rows keep what they held
            kbs = H // 64
            pad_rows = np.arange(T, full.shape[0])
            for rr in pad_rows[:3]:
                base = ((rr // 128) * kbs) * 512 + (rr % 32) * 16 + (rr % 128) // 32 * 4
                assert (got[base:base + 4] == 0xA5).all()
        else:
            assert np.array_equal(got.reshape(T, H // 16), wsc)
    elif quant == NVFP4_QUANT_E4M3:
        wc, wsc = e4m3_rows(want_y)
        assert torch.equal(codes[:T].cpu(), wc)
        assert np.array_equal(scales[:T].cpu().numpy(), wsc)
        assert (codes[T] == 0xA5).all() and (scales[T] == -3.0).all()


QUANTS = [(NVFP4_QUANT_NONE, 0), (NVFP4_QUANT_NVFP4, NVFP4_SCALES_ROWMAJOR), (NVFP4_QUANT_NVFP4, NVFP4_SCALES_MMA),
          (NVFP4_QUANT_E4M3, 0)]


@pytest.mark.parametrize("quant,layout", QUANTS)
@pytest.mark.parametrize("T,H", [(1, 64), (1, 7168), (3, 128), (5, 576), (64, 7168), (129, 1536), (300, 512),
                                 (17, 4096), (2, 16384), (1, 32768), (257, 64), (150, 8256), (1000, 1024)])
def test_shapes(T, H, quant, layout):
    check(T, H, quant, layout, seed=T + H)


@pytest.mark.parametrize("H", [16, 32, 48, 80, 112, 144, 208, 1008, 7152, 8208, 16400, 32752])
@pytest.mark.parametrize("quant", [NVFP4_QUANT_NONE, NVFP4_QUANT_NVFP4, NVFP4_QUANT_E4M3])
def test_odd_widths(H, quant):
    """Widths that are no multiple of a scale group, a warp or a thread's share."""
    check(7, H, quant, seed=H)


@pytest.mark.parametrize("quant,layout", QUANTS)
@pytest.mark.parametrize("res", [True, False])
def test_strided_rows(quant, layout, res):
    check(37, 832, quant, layout, res=res, pads=(8, 64, 24, 40), seed=3)


@pytest.mark.parametrize("quant,layout", QUANTS[1:])
def test_without_bf16_output(quant, layout):
    check(9, 1536, quant, layout, y=False, seed=4)


@pytest.mark.parametrize("res", [True, False])
def test_many_rows(res):
    """More rows than blocks that fit on the device at once, the last group of rows partial."""
    check(4099, 256, NVFP4_QUANT_NVFP4, res=res, seed=5)
    check(2053, 2048, NVFP4_QUANT_E4M3, res=res, seed=6)


def test_special_rows():
    """Rows of zeros, of the smallest and the largest values, cancelling sums,
    and a row whose neighbours are not finite."""
    T, H = 8, 256
    x, r = rows(T, H, 1), rows(T, H, 2)
    x[0], r[0] = 0.0, 0.0
    x[1], r[1] = -0.0, -0.0
    x[2], r[2] = 1e-38, 0.0
    x[3], r[3] = 3e38 / 256, 0.0
    r[4] = -x[4]                                        # h = 0 although x and residual are not
    x[5], r[5] = 1e-20, -1e-20
    for quant in (NVFP4_QUANT_NONE, NVFP4_QUANT_NVFP4, NVFP4_QUANT_E4M3):
        check(T, H, quant, x=x, r=r)
    y = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    clean = torch.empty_like(y)
    w = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    nvfp4_add_rmsnorm(x.to(DEV), w, EPS, y=clean)
    bad = x.clone()
    bad[2, 5], bad[6, 0] = float("nan"), float("inf")
    nvfp4_add_rmsnorm(bad.to(DEV), w, EPS, y=y)
    keep = [0, 1, 3, 4, 5, 7]
    assert torch.equal(bits(y[keep]), bits(clean[keep]))


def test_zero_eps():
    x = rows(5, 320, 9)
    w = torch.ones(320, dtype=torch.bfloat16)
    y = torch.empty(5, 320, dtype=torch.bfloat16, device=DEV)
    nvfp4_add_rmsnorm(x.to(DEV), w.to(DEV), 0.0, y=y)
    _, want = reference(x, None, w, 0.0)
    assert torch.equal(bits(y), bits(torch.from_numpy(want).to(torch.bfloat16)))


@pytest.mark.parametrize("T,H", [(70, 7168), (2000, 512)])
def test_in_place(T, H):
    """residual_out = residual and y = x; residual_out = x and y = residual."""
    x, r = rows(T, H, 1), rows(T, H, 2)
    w = torch.ones(H, dtype=torch.bfloat16)
    h, y = reference(x, r, w)
    y = torch.from_numpy(y).to(torch.bfloat16)
    for swap in (False, True):
        xd, rd = x.to(DEV), r.to(DEV)
        ro, yo = (xd, rd) if swap else (rd, xd)
        nvfp4_add_rmsnorm(xd, w.to(DEV), EPS, y=yo, residual=rd, residual_out=ro)
        assert torch.equal(bits(ro), bits(h)) and torch.equal(bits(yo), bits(y))


def test_empty_batch():
    e = torch.empty(0, 256, dtype=torch.bfloat16, device=DEV)
    nvfp4_add_rmsnorm(e, torch.ones(256, dtype=torch.bfloat16, device=DEV), EPS, y=e)
    torch.cuda.synchronize()


def test_rows_do_not_depend_on_the_batch():
    """A row's bits are the same alone, in a small batch and in a large one."""
    H = 7168
    x, r = rows(600, H, 11).to(DEV), rows(600, H, 12).to(DEV)
    w = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    gs = torch.tensor([60.0], device=DEV)

    def run(a, b):
        n = b - a
        out = [torch.empty(n, H, dtype=torch.bfloat16, device=DEV), torch.empty(n, H, dtype=torch.bfloat16, device=DEV),
               torch.empty(n, H // 2, dtype=torch.uint8, device=DEV), torch.empty(n, H // 16, dtype=torch.uint8, device=DEV)]
        nvfp4_add_rmsnorm(x[a:b], w, EPS, y=out[0], residual=r[a:b], residual_out=out[1], quant=NVFP4_QUANT_NVFP4, gs=gs,
                          codes=out[2], scales=out[3])
        return out
    whole = run(0, 600)
    for a, b in ((0, 1), (599, 600), (100, 140), (7, 300)):
        for got, want in zip(run(a, b), whole):
            assert torch.equal(got, want[a:b])


def test_graph_replay_and_side_stream():
    T, H = 33, 1536
    x, r = rows(T, H, 1).to(DEV), rows(T, H, 2).to(DEV)
    w = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    codes = torch.empty(T, H, dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.empty(T, H // 128, device=DEV)
    ro, y = torch.empty_like(x), torch.empty_like(x)

    def call(stream=None):
        nvfp4_add_rmsnorm(x, w, EPS, y=y, residual=r, residual_out=ro, quant=NVFP4_QUANT_E4M3, codes=codes, scales=scales,
                          stream=stream)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (5, 6):
        x.copy_(rows(T, H, seed))
        graph.replay()
        torch.cuda.synchronize()
        h, want = reference(x.cpu(), r.cpu(), w.cpu())
        assert torch.equal(bits(ro), bits(h))
        assert torch.equal(codes.cpu().view(torch.uint8), e4m3_rows(want)[0])
    side = torch.cuda.Stream()
    x.copy_(rows(T, H, 7))
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    side.synchronize()
    assert torch.equal(bits(ro), bits(reference(x.cpu(), r.cpu(), w.cpu())[0]))


def test_binding_refusals():
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(256, dtype=torch.bfloat16, device=DEV)
    c = torch.zeros(4, 128, dtype=torch.uint8, device=DEV)
    s = torch.zeros(64, dtype=torch.uint8, device=DEV)
    gs = torch.ones(1, device=DEV)
    q = dict(quant=NVFP4_QUANT_NVFP4, gs=gs, codes=c, scales=s)
    bad = [
        (dict(weight=w[:-1]), "weight must hold"), (dict(weight=w.float()), "weight must be torch.bfloat16"),
        (dict(y=None), "y is required"), (dict(y=x[:3]), "y must be"), (dict(y=x.t()), "y must be"),
        (dict(residual=x), "come together"), (dict(residual_out=x), "come together"),
        (dict(residual=x[:2], residual_out=x), "residual must be"), (dict(x=x.float()), "x must be torch.bfloat16"),
        (dict(q, gs=None), "gs is required"), (dict(q, codes=None), "codes is required"),
        (dict(q, codes=c[:3]), "codes must hold"), (dict(q, scales=s[:60]), "scales must hold"),
        (dict(q, scales=s, scale_layout=NVFP4_SCALES_MMA), "scales must hold"),
        (dict(q, codes=c.cpu()), "CUDA tensor"), (dict(weight=w.cpu()), "CUDA tensor"),
        (dict(quant=NVFP4_QUANT_E4M3, codes=c, scales=gs), "codes must hold"),
        (dict(x=x[:, ::2], weight=w[:128], y=x[:, :128]), "unit stride"),
    ]
    for change, match in bad:
        args = dict(x=x, weight=w, eps=EPS, y=x)
        args.update(change)
        with pytest.raises(ValueError, match=match):
            nvfp4_add_rmsnorm(**args)


@pytest.mark.parametrize("H", [128, 208, 7168])
@pytest.mark.parametrize("low", [2.0 ** -126, 2.0 ** -118, 1e-36, 2.0 ** -100, 2.0 ** -99])
def test_e4m3_groups_of_tiny_values(H, low):
    """Groups whose largest magnitude is so small that 448 / a is not an fp32
    number, zeros among them (a dead channel group beside live ones): each
    code is E4M3 of y * 448 / a, taken here in 64 bits.  The quotient and the
    product each round by 2^-24, so a code is one of the two E4M3 neighbours
    of a value within that of a border between them."""
    T = 6
    x = rows(T, H, 3)
    w = torch.ones(H, dtype=torch.bfloat16)
    dead = slice(0, 128) if H > 128 else slice(0, 0)     # (one group alone: the weight is small instead)
    g = torch.Generator().manual_seed(1)
    tiny = (torch.randn(H, generator=g) * low).to(torch.bfloat16)
    tiny[::3] = 0.0
    if H > 128:
        x[:, dead] = tiny[dead]
        x[1, dead] = 0.0
    else:
        w = tiny
    codes = torch.empty(T, H, dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.empty(T, (H + 127) // 128, device=DEV)
    nvfp4_add_rmsnorm(x.to(DEV), w.to(DEV), EPS, quant=NVFP4_QUANT_E4M3, codes=codes, scales=scales)
    _, y = reference(x, None, w)
    got = codes.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    for i in range(0, H, 128):
        v = y[:, i:i + 128].astype(np.float64)
        a = np.abs(v).max(axis=1, keepdims=True)
        assert np.array_equal(scales[:, i // 128].cpu().numpy(), (y[:, i:i + 128].__abs__().max(axis=1) / np.float32(448.0)))
        want = v * np.where(a > 0, 448.0 / np.where(a > 0, a, 1), 0)
        for sign in (-1, 1):                             # one of the codes of want (1 -+ 2^-22)
            near = torch.from_numpy(want * (1 + sign * 2.0 ** -22)).clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
            side = near if sign < 0 else np.where(got[:, i:i + 128] == side, side, near)
        assert np.array_equal(got[:, i:i + 128], side)
