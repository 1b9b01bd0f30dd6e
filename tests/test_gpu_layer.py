"""The operators around the routed block in the order a layer runs them."""
import numpy as np
import pytest
import torch

import oracle as O
from nvfp4_moe_expert_topk_b200 import (NVFP4_QUANT_NVFP4, NVFP4_SCALES_MMA, NVFP4_SCORING_SIGMOID, nvfp4_add_rmsnorm,
                                        nvfp4_gemm, nvfp4_gemv, nvfp4_moe_balance, nvfp4_moe_balance_backward,
                                        nvfp4_moe_balance_workspace_size, nvfp4_moe_forward, nvfp4_moe_forward_quantized,
                                        nvfp4_moe_get_error, nvfp4_moe_topk, nvfp4_scales_bytes)
from nvfp4_moe_expert_topk_b200 import prep
from nvfp4_moe_expert_topk_b200 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Layer:
    """norm -> router -> routed experts on the norm's NVFP4 rows, on the tiny
    workload's weights; everything allocated once."""

    def __init__(self, T):
        self.cfg = cfg = W.MOE_CONFIGS["tiny"]
        self.T = T
        g = torch.Generator().manual_seed(T)
        H, E, k = cfg.H, cfg.E, cfg.k
        self.wts = prep.MoeWeights.synthetic(cfg, DEV)
        self.inter_gs = torch.full((E,), 200.0, device=DEV)
        self.x = torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV)
        self.res = torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV)
        self.w = (1 + 0.1 * torch.randn(H, generator=g)).to(torch.bfloat16).to(DEV)
        self.router = (torch.randn(H, E, generator=g) / H ** 0.5).to(DEV)
        self.gs = torch.tensor([2688.0 / 5.0], device=DEV)
        self.res_out, self.y = torch.empty_like(self.x), torch.empty_like(self.x)
        self.codes = torch.empty(T, H // 2, dtype=torch.uint8, device=DEV)
        self.scales = torch.empty(T, H // 16, dtype=torch.uint8, device=DEV)
        self.logits = torch.empty(T, E, device=DEV)
        self.ids = torch.empty(T, k, dtype=torch.int32, device=DEV)
        self.weights = torch.empty(T, k, device=DEV)
        self.out = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
        self.ws = prep.workspace(T, k, E, H, cfg.I, DEV)
        self.counts = torch.empty(1, E, dtype=torch.int32, device=DEV)
        self.tokens = torch.empty(1, dtype=torch.int32, device=DEV)
        self.probs, self.loss = torch.empty(1, E, device=DEV), torch.empty(1, device=DEV)
        self.bws = torch.empty(nvfp4_moe_balance_workspace_size(T, 1, E), dtype=torch.uint8, device=DEV)
        self.grad = torch.empty(T, E, device=DEV)

    def run(self):
        cfg = self.cfg
        nvfp4_add_rmsnorm(self.x, self.w, 1e-6, y=self.y, residual=self.res, residual_out=self.res_out,
                          quant=NVFP4_QUANT_NVFP4, gs=self.gs, codes=self.codes, scales=self.scales)
        torch.matmul(self.y.float(), self.router, out=self.logits)
        nvfp4_moe_topk(self.logits, cfg.k, self.ids, self.weights, NVFP4_SCORING_SIGMOID)
        nvfp4_moe_forward_quantized(self.codes, self.scales, self.ids, self.weights, self.gs, **self.wts.args(),
                                    inter_gs=self.inter_gs, out=self.out, workspace=self.ws)
        nvfp4_moe_balance(self.logits, self.ids, cfg.k, self.counts, self.tokens, self.probs, self.loss, self.bws,
                          scoring=NVFP4_SCORING_SIGMOID)
        nvfp4_moe_balance_backward(self.logits, self.ids, cfg.k, self.counts, self.tokens, self.loss, self.grad,
                                   scoring=NVFP4_SCORING_SIGMOID)


@pytest.mark.parametrize("T", [1, 64, 200])
def test_norm_feeds_the_routed_block(T):
    """The forward on the norm's NVFP4 rows equals the forward on its bf16
    rows, bit for bit; the counts are the forward's own routing's."""
    m = Layer(T)
    m.run()
    want = torch.empty_like(m.out)
    ws = prep.workspace(T, m.cfg.k, m.cfg.E, m.cfg.H, m.cfg.I, DEV)
    nvfp4_moe_forward(m.y, m.ids, m.weights, m.gs, **m.wts.args(), inter_gs=m.inter_gs, out=want, workspace=ws)
    torch.cuda.synchronize()
    assert nvfp4_moe_get_error(m.ws) == 0
    assert torch.isfinite(m.out.float()).all() and m.out.float().abs().max() > 0
    assert torch.equal(m.out.view(torch.int16), want.view(torch.int16))
    assert np.array_equal(m.counts[0].cpu().numpy(), np.bincount(m.ids.cpu().numpy().ravel(), minlength=m.cfg.E))
    assert int(m.tokens) == T


def test_layer_replayed_from_a_graph():
    """The whole run in one CUDA graph, on new inputs, equals the eager run."""
    m = Layer(96)
    m.run()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        m.run()
    for seed in (1, 2):
        g = torch.Generator().manual_seed(seed)
        m.x.copy_(torch.randn(96, m.cfg.H, generator=g).to(torch.bfloat16))
        m.res.copy_(torch.randn(96, m.cfg.H, generator=g).to(torch.bfloat16))
        m.run()
        want = [t.clone() for t in (m.y, m.out, m.counts, m.loss, m.grad, m.res_out)]
        for t in (m.y, m.out, m.counts, m.loss, m.grad, m.res_out):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((m.y, m.out, m.counts, m.loss, m.grad, m.res_out), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T", [3, 130])
def test_norm_feeds_the_projection(T):
    """The norm's MMA-layout rows go straight into nvfp4_gemm: the same bits as
    quantising its bf16 rows first; its bf16 rows go into nvfp4_gemv."""
    H, N = 1536, 384
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV)
    b = (0.02 * torch.randn(N, H, generator=g)).to(torch.bfloat16).to(DEV)
    bc, bs, bg = prep.quantize(b)
    w = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    gs = torch.tensor([2688.0 / 6.0], device=DEV)
    y = torch.empty_like(x)
    codes = torch.empty(T, H // 2, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(nvfp4_scales_bytes(T, H, NVFP4_SCALES_MMA), dtype=torch.uint8, device=DEV)
    nvfp4_add_rmsnorm(x, w, 1e-6, y=y, quant=NVFP4_QUANT_NVFP4, gs=gs, codes=codes, scales=scales,
                      scale_layout=NVFP4_SCALES_MMA)
    out, want = (torch.empty(T, N, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    nvfp4_gemm(codes, scales, gs, bc, bs, bg, [N], out)
    qc, qs, _ = prep.quantize(y, gs)
    nvfp4_gemm(qc, qs, gs, bc, bs, bg, [N], want)
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    few = torch.empty(min(T, 16), N, dtype=torch.bfloat16, device=DEV)
    nvfp4_gemv(y[:16], bc, bs, bg, [N], few)
    # the two differ by the quantisation of the activations only
    ref = O.dequantize(bc.cpu().numpy(), _rowmajor(bs, N, H), np.float32(bg.item())).astype(np.float64)
    exact = y[:16].double().cpu().numpy() @ ref.T
    got = few.double().cpu().numpy()
    assert np.linalg.norm(got - exact) <= 2.0 ** -8 * np.linalg.norm(exact)
    assert np.linalg.norm(out[:16].double().cpu().numpy() - exact) <= 0.2 * np.linalg.norm(exact)


def _rowmajor(scales, rows, cols):
    from helpers import from_mma_layout
    return from_mma_layout(scales.cpu().numpy(), rows, cols)
