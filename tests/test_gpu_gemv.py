"""nvfp4_gemv against the product of the dequantised weights in 64 bits.

Tolerance, derived from the arithmetic: the weights e2m1 * e4m3 and their
products with bf16 are exact in fp32; an output is a sum of K products, in
which no term passes more than K / 8 + 32 fp32 additions (each within 2^-23 of
its operands' magnitudes, the tensor cores' truncation included), then one
division (2^-24) and one rounding to bf16 (2^-8 of the value):
  |err| <= (K / 8 + 33) * 2^-23 * sum_k |x w| / gs + 2^-8 |out|."""
import numpy as np
import pytest
import torch

import oracle as O
from helpers import to_mma_layout
from nvfp4_moe_expert_topk_b200 import NVFP4_SCALES_MMA, Nvfp4Error, nvfp4_gemm, nvfp4_gemv
from nvfp4_moe_expert_topk_b200 import prep

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Weights:
    """Random NVFP4 weights: every code, scales over `span` of the E4M3 range."""

    def __init__(self, N, K, seed, seg=None, span=(8, 0x7E)):
        rng = np.random.default_rng(seed)
        self.N, self.K = N, K
        self.seg = list(seg or [N])
        self.codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
        self.scales = rng.integers(span[0], span[1] + 1, (N, K // 16)).astype(np.uint8)
        self.gs = (rng.uniform(0.5, 3000.0, len(self.seg))).astype(np.float32)

    def dev(self):
        return (torch.from_numpy(self.codes).to(DEV), torch.from_numpy(to_mma_layout(self.scales)).to(DEV),
                torch.from_numpy(self.gs).to(DEV), self.seg)

    def values(self):
        """Dequantised in 64 bits, without the global scales; and those per row."""
        v = O.dequantize(self.codes, self.scales, np.float32(1.0)).astype(np.float64)
        g = np.repeat(self.gs.astype(np.float64), np.diff([0] + self.seg))
        return v, g


def check(M, N, K, seed=0, seg=None, x=None, ldx=0, ldo=0, w=None):
    w = w or Weights(N, K, seed, seg)
    if x is None:
        x = torch.randn(M, K, generator=torch.Generator().manual_seed(seed + 1)).to(torch.bfloat16)
    codes, scales, gs, ends = w.dev()
    xb = torch.full((M, K + ldx), 3.0, dtype=torch.bfloat16, device=DEV)
    xb[:, :K] = x.to(DEV)
    ob = torch.full((M + 1, N + ldo), 55.0, dtype=torch.bfloat16, device=DEV)
    nvfp4_gemv(xb[:, :K], codes, scales, gs, ends, ob[:M, :N])
    first = ob.clone()
    nvfp4_gemv(xb[:, :K], codes, scales, gs, ends, ob[:M, :N])
    torch.cuda.synchronize()
    assert torch.equal(first.view(torch.int16), ob.view(torch.int16))       # the same bits again
    assert (ob[M] == 55.0).all() and (ob[:, N:] == 55.0).all()
    v, g = w.values()
    xd = x.double().numpy()
    want = (xd @ v.T) / g
    mag = (np.abs(xd) @ np.abs(v).T) / g
    got = ob[:M, :N].double().cpu().numpy()
    tol = (K / 8 + 33) * 2.0 ** -23 * mag + 2.0 ** -8 * np.abs(want) + 1e-38
    worst = (np.abs(got - want) / tol).max()
    assert worst <= 1.0, worst
    return got


@pytest.mark.parametrize("M", list(range(1, 17)))
def test_row_counts(M):
    check(M, 264, 448, seed=M)


@pytest.mark.parametrize("N,K", [(1, 64), (7, 64), (31, 128), (32, 192), (33, 256), (127, 320), (128, 64), (129, 576),
                                 (200, 256), (1000, 1536), (2048, 7168), (384, 8192), (4100, 64), (65, 16384)])
@pytest.mark.parametrize("M", [1, 5, 8, 9, 16])
def test_sizes(M, N, K):
    check(M, N, K, seed=N + K)


@pytest.mark.parametrize("seg", [[1, 200], [7, 31, 199, 200], [128, 200], [32, 64, 96, 200], [199, 200]])
def test_segments(seg):
    """Global scales change at any row, inside a tile too."""
    check(3, 200, 256, seed=9, seg=seg)
    check(12, 200, 256, seed=9, seg=seg)


@pytest.mark.parametrize("M", [1, 2, 11])
def test_strides(M):
    check(M, 130, 320, seed=2, ldx=8, ldo=1)
    check(M, 130, 320, seed=2, ldx=72, ldo=7)


@pytest.mark.parametrize("M,K", [(1, 64), (4, 448), (16, 2048)])
def test_one_hot_rows_are_exact(M, K):
    """x = 2^p at one column: the output is that weight, rounded once.  Covers
    nibble order, scale placement and the column order of the products."""
    N = 160
    w = Weights(N, K, 5, span=(0, 0x7E))                 # subnormal and zero scales too
    w.gs[:] = 1.0
    v, _ = w.values()
    rng = np.random.default_rng(6)
    for trial in range(12):
        cols = rng.integers(0, K, M)
        x = torch.zeros(M, K, dtype=torch.bfloat16)
        p = 2.0 ** rng.integers(-20, 21, M)
        x[torch.arange(M), torch.from_numpy(cols)] = torch.from_numpy(p).to(torch.bfloat16)
        got = check(M, N, K, w=w, x=x)
        want = torch.from_numpy(v[:, cols].T * p[:, None]).to(torch.bfloat16).double().numpy()
        assert np.array_equal(got, want)


@pytest.mark.parametrize("M,N,K", [(1, 96, 1024), (7, 224, 512), (16, 64, 8192)])
def test_whole_number_sums_are_exact(M, N, K):
    """Small whole x and unit scales: every partial sum is exact in fp32, so
    the output is the exact sum rounded once, whatever the order."""
    w = Weights(N, K, 7, span=(0x38, 0x38))              # scale 1.0
    w.gs[:] = 1.0
    x = torch.randint(-2, 3, (M, K), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    got = check(M, N, K, w=w, x=x)
    v, _ = w.values()
    want = torch.from_numpy(x.double().numpy() @ v.T).to(torch.bfloat16).double().numpy()
    assert np.array_equal(got, want)


@pytest.mark.parametrize("seed", range(16))
def test_random_shapes(seed):
    rng = np.random.default_rng(300 + seed)
    M, N, K = int(rng.integers(1, 17)), int(np.exp(rng.uniform(0, 8.3))), 64 * int(np.exp(rng.uniform(0, 4.2)))
    cuts = sorted(set(int(v) for v in rng.integers(1, N + 1, 3)) | {N})
    check(M, N, K, seed=seed, seg=cuts, ldx=8 * int(rng.integers(0, 3)), ldo=int(rng.integers(0, 5)))


@pytest.mark.parametrize("M", [2, 8, 16])
def test_long_k(M):
    """More columns than the block holds of x at a time."""
    check(M, 70, 131072 + 64, seed=1)


def test_extreme_values():
    """Activations over the whole bf16 range; zero rows; a row that is not
    finite spoils only itself."""
    M, N, K = 6, 96, 512
    w = Weights(N, K, 3, span=(0, 0x7E))
    g = torch.Generator().manual_seed(2)
    x = (torch.randn(M, K, generator=g) * torch.exp2(torch.randint(-60, 60, (M, K), generator=g).float())).to(torch.bfloat16)
    x[1] = 0.0
    x[2] = (torch.randn(K, generator=g) * 2.0 ** -120).to(torch.bfloat16)
    x[3, ::2] = 0.0
    check(M, N, K, w=w, x=x)
    codes, scales, gs, ends = w.dev()
    clean = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    out = torch.empty_like(clean)
    nvfp4_gemv(x.to(DEV), codes, scales, gs, ends, clean)
    bad = x.clone()
    bad[4, 7], bad[5, 0] = float("nan"), float("inf")
    nvfp4_gemv(bad.to(DEV), codes, scales, gs, ends, out)
    assert torch.equal(out[:4].view(torch.int16), clean[:4].view(torch.int16))


def test_rows_do_not_depend_on_their_neighbours():
    """Each row's bits are those of the other rows' absence or permutation
    within the same row count."""
    N, K, M = 300, 1024, 8
    w = Weights(N, K, 4)
    codes, scales, gs, ends = w.dev()
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).to(DEV)
    out = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    nvfp4_gemv(x, codes, scales, gs, ends, out)
    perm = torch.tensor([3, 1, 7, 0, 2, 6, 5, 4], device=DEV)
    out2 = torch.empty_like(out)
    nvfp4_gemv(x[perm].contiguous(), codes, scales, gs, ends, out2)
    assert torch.equal(out2.view(torch.int16), out[perm].view(torch.int16))


def test_empty_and_refused():
    w = Weights(64, 128, 1)
    codes, scales, gs, ends = w.dev()
    e = torch.empty(0, 128, dtype=torch.bfloat16, device=DEV)
    nvfp4_gemv(e, codes, scales, gs, ends, torch.empty(0, 64, dtype=torch.bfloat16, device=DEV))
    x = torch.zeros(17, 128, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(Nvfp4Error) as err:
        nvfp4_gemv(x, codes, scales, gs, ends, torch.empty(17, 64, dtype=torch.bfloat16, device=DEV))
    assert err.value.status == -2
    x = x[:2]
    o = torch.empty(2, 64, dtype=torch.bfloat16, device=DEV)
    for change, match in [(dict(out=o[:1]), "out must be"), (dict(x=x.float()), "x must be"), (dict(b_codes=codes[:, :8]), "b_codes must"),
                          (dict(b_scales=scales[:100]), "b_scales must hold"), (dict(b_gs=gs.expand(2)), "b_gs must"),
                          (dict(b_codes=codes.cpu()), "CUDA tensor"), (dict(out=o.float()), "out must be torch.bfloat16"),
                          (dict(x=x.t()[:2, :2]), "x must have unit stride|out must be")]:
        args = dict(x=x, b_codes=codes, b_scales=scales, b_gs=gs, seg_end=ends, out=o)
        args.update(change)
        with pytest.raises((ValueError, Nvfp4Error), match=match):
            nvfp4_gemv(**args)


def test_graph_replay_and_side_stream():
    M, N, K = 5, 512, 2048
    w = Weights(N, K, 2)
    codes, scales, gs, ends = w.dev()
    x = torch.randn(M, K).to(torch.bfloat16).to(DEV)
    out, want = (torch.empty(M, N, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    nvfp4_gemv(x, codes, scales, gs, ends, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nvfp4_gemv(x, codes, scales, gs, ends, out)
    for _ in range(2):
        x.copy_(torch.randn(M, K).to(torch.bfloat16))
        graph.replay()
        nvfp4_gemv(x, codes, scales, gs, ends, want)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    nvfp4_gemv(x, codes, scales, gs, ends, out, stream=side)
    side.synchronize()
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))


def test_same_weights_as_the_dense_gemm():
    """One set of weights serves both: against nvfp4_gemm on activations that
    NVFP4 holds exactly, the two differ by their roundings only."""
    M, N, K = 8, 256, 512
    g = torch.Generator().manual_seed(3)
    x = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])[torch.randint(0, 8, (M, K), generator=g)]
    x[:, ::16] = 6.0                                     # every block's scale is then the same power
    x = (x * torch.randint(0, 2, (M, K), generator=g).mul(2).sub(1)).to(torch.bfloat16).to(DEV)
    b = (0.02 * torch.randn(N, K, generator=g)).to(torch.bfloat16).to(DEV)
    bc, bs, bg = prep.quantize(b)
    ac, asc, ag = prep.quantize(x, torch.tensor([448.0], device=DEV))
    dense = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    few = torch.empty_like(dense)
    nvfp4_gemm(ac, asc, ag, bc, bs, bg, [N], dense)
    nvfp4_gemv(x, bc, bs, bg, [N], few)
    d, f = dense.double(), few.double()
    mag = x.double().abs() @ b.double().abs().t()
    assert ((d - f).abs() <= 2 * 2.0 ** -8 * d.abs() + 2 * (K / 8 + 33) * 2.0 ** -23 * 1.3 * mag).all()


@pytest.mark.parametrize("M,N,K", [(1, 96, 64), (1, 2048, 7168), (3, 200, 256), (8, 130, 1984), (9, 33, 512), (16, 264, 448),
                                   (5, 4100, 2048), (2, 70, 131072 + 64)])
@pytest.mark.parametrize("top", [32, 45, 126])
def test_large_values_on_zero_weights(M, N, K, top):
    """Activations of 2^top whose weights are zero (by their code or by their
    block's scale) beside ordinary ones and ones far below 1: what is left
    of the sum comes from the small ones, so that the bound says whether they
    were held."""
    w = Weights(N, K, N + K)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(K)).to(torch.bfloat16)
    x[:, 16:32] *= 2.0 ** -30
    big = [0, 1, 17, 40, K - 1, K - 20]
    for i, c in enumerate(big):
        x[i % M, c] = 2.0 ** top * (1 if i % 2 else -1)
        w.codes[:, c // 2] &= 0x0F if c % 2 else 0xF0    # code 0 in the column
    w.scales[:, 3] = 0                                   # and a whole block by its scale
    x[M - 1, 48:52] = 2.0 ** top
    w.codes[N // 2:, 16:] = 0                            # rows of only the smallest activations
    check(M, N, K, w=w, x=x)


@pytest.mark.parametrize("M", [1, 6, 16])
def test_bands_of_magnitudes(M):
    """Activations of very different magnitudes, each output made of one of
    them alone: 2^-126 .. 2^100, subnormal ones beside them."""
    N, K = 160, 640
    w = Weights(N, K, 12)
    keep = np.zeros((N, K), bool)
    bands = np.arange(K) // 64                           # 10 bands of 64 columns
    for n in range(N):
        keep[n] = bands == n % 10
    w.codes &= (np.where(keep[:, 0::2], 0x0F, 0) | np.where(keep[:, 1::2], 0xF0, 0)).astype(np.uint8)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(M)).double()
    p = np.array([100, 70, 37, 5, 0, -30, -61, -93, -110, -118])
    x = (x * torch.from_numpy(2.0 ** p[bands])).to(torch.bfloat16)
    got = check(M, N, K, w=w, x=x)
    assert (np.abs(got[:, np.arange(N) % 10 < 9]).max(axis=1) > 0).all()
    x[:, 64:] = 0.0                                      # one band alone, then the whole range in one row only
    check(M, N, K, w=w, x=x)


@pytest.mark.parametrize("M,N,K", [(16, 65536, 1536), (5, 7168, 8192), (1, 384, 1024)])
def test_a_wait_that_gives_up_is_seen(M, N, K):
    """Weights that do not come within the wait's bound: the outputs they have
    a share in are NaN, never partial sums; all others are as ever, and so is
    the next call."""
    import time
    from nvfp4_moe_expert_topk_b200 import nvfp4_debug_gemv_timeout
    g = torch.Generator(device=DEV).manual_seed(N)
    x = torch.randn(M, K, generator=g, device=DEV).to(torch.bfloat16)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.randint(8, 120, ((N + 127) // 128 * 128 * (K // 16),), generator=g, device=DEV, dtype=torch.uint8)
    gs = torch.tensor([3.0], device=DEV)
    want, got = (torch.empty(M, N, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    nvfp4_gemv(x, codes, scales, gs, [N], want)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    nvfp4_debug_gemv_timeout(x, codes, scales, gs, [N], got)
    torch.cuda.synchronize()
    assert 1.5 < time.perf_counter() - t0 < 30.0
    lost = torch.isnan(got)
    assert not torch.isnan(want).any()
    n = torch.arange(N, device=DEV)
    first = (n < 128) & (n % 32 < 8)
    assert lost[:, first].all()                          # the tile whose copy was withheld
    assert (lost == lost[:1]).all() and lost.float().mean() < 0.2
    assert torch.equal(got[~lost].view(torch.int16), want[~lost].view(torch.int16))
    nvfp4_gemv(x, codes, scales, gs, [N], got)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
