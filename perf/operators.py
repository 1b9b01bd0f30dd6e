"""The operators around the routed-expert block, and the cases they are measured on.

- norm: residual addition + RMS norm with a quantised output (the step in
  front of the router, the MoE block and the projections);
- gemv: products of a few bf16 rows with NVFP4 weights (the projections while
  few sequences are decoded);
- balance: per-expert counts and the load-balance loss of the router, its
  gradient and the gradient of the top-k weights.

`run` computes them in elementary torch operations when `own` is false and
through the library's entry points when it is true.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one sequence decoding: the row in front of the MoE block of the 7168-wide model (latency)
        dict(name="norm_row1_nvfp4", op="norm", T=1, H=7168, res=True, quant="nvfp4", layout="rows"),
        # the decode batch of 64 tokens, 8-bit rows
        dict(name="norm_decode64_e4m3", op="norm", T=64, H=7168, res=True, quant="e4m3", layout="rows"),
        # the norm of the 1536-wide compressed query, whose NVFP4 rows feed the q_b GEMM; a ragged batch, no residual
        dict(name="norm_qlora2041_mma", op="norm", T=2041, H=1536, res=False, quant="nvfp4", layout="mma"),
        # the prefill batch in front of the MoE block
        dict(name="norm_prefill4096_nvfp4", op="norm", T=4096, H=7168, res=True, quant="nvfp4", layout="rows"),
        # a small odd matrix (fewer rows than one scale block of 128 past the first): latency
        dict(name="gemv_small", op="gemv", M=3, N=200, K=256, segs=1),
        # one token through fused_wqa_wkv (two global scales)
        dict(name="gemv_wqa_wkv_1", op="gemv", M=1, N=2048, K=7168, segs=2),
        # five sequences through o_b
        dict(name="gemv_o_b_5", op="gemv", M=5, N=7168, K=8192, segs=1),
        # sixteen sequences through q_b, the largest projection
        dict(name="gemv_q_b_16", op="gemv", M=16, N=65536, K=1536, segs=1),
        # load statistics of a decode batch on one expert-parallel slice
        dict(name="balance_decode64", op="balance", do="loss", T=64, E=48, k=6, S=1, scoring="sigmoid", pad=False),
        # the prefill batch: ragged sequences with padded tokens
        dict(name="balance_prefill4096", op="balance", do="loss", T=4096, E=384, k=6, S=7, scoring="softmax", pad=True),
        # its gradient, with the gradient of the top-k weights
        dict(name="balance_grad4096", op="balance", do="grad", T=4096, E=384, k=6, S=7, scoring="sigmoid", pad=True),
        # a training step of the router over a long batch: loss, then gradient
        dict(name="balance_step65536", op="balance", do="step", T=65536, E=384, k=6, S=33, scoring="softmax", pad=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "gemv", "balance"])
    if op == "norm":
        quant = rng.choice(["none", "nvfp4", "e4m3"])
        layout = rng.choice(["rows", "mma"]) if quant == "nvfp4" else "rows"
        unit = 64 if layout == "mma" else 16
        H = unit * _log(rng, 64 // unit, 16384 // unit)
        T = _log(rng, 1, min(8192, 4096 * 7168 // H))
        return dict(op=op, T=T, H=H, res=rng.random() < 0.7, quant=quant, layout=layout)
    if op == "gemv":
        K = 64 * _log(rng, 1, 128)
        N = _log(rng, 1, min(65536, 65536 * 1536 // K))
        return dict(op=op, M=rng.randint(1, 16), N=N, K=K, segs=2 if N >= 64 and rng.random() < 0.4 else 1)
    E = _log(rng, 2, 1024)
    T = _log(rng, 1, min(65536, 65536 * 384 // E))
    return dict(op=op, do=rng.choice(["loss", "grad", "step"]), T=T, E=E, k=rng.randint(1, min(E, 12)), S=_log(rng, 1, 64),
                scoring=rng.choice(["softmax", "sigmoid"]), pad=rng.random() < 0.5)


def work(case):
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        b = 2 * T * H + 2 * H + 2 * T * H                     # x, weight, y
        if case["res"]:
            b += 4 * T * H                                    # residual read, sum written
        if case["quant"] == "nvfp4":
            b += T * H // 2 + T * H // 16
        elif case["quant"] == "e4m3":
            b += T * H + 4 * T * ((H + 127) // 128)
        return {"bytes": b, "flops": 5 * T * H}
    if case["op"] == "gemv":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": N * K // 2 + N * K // 16 + 2 * M * K + 2 * M * N, "flops": 2 * M * N * K}
    T, E, k, S = case["T"], case["E"], case["k"], case["S"]
    loss = 4 * T * E + 4 * T * k + 8 * S * E
    grad = 8 * T * E + 8 * T * k + 4 * S * E
    if case["do"] == "loss":
        return {"bytes": loss, "flops": 6 * T * E}
    if case["do"] == "grad":
        return {"bytes": grad, "flops": 10 * T * E}
    return {"bytes": loss + grad, "flops": 16 * T * E}


# ---------------------------------------------------------------- number formats
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _e2m1_codes(v):
    """Codes of fp32 values, nearest, ties to the even code, saturating at 6."""
    a = v.abs()
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return c + 8 * torch.signbit(v).to(torch.uint8)


def _nvfp4(y, gs):
    """y fp32 [rows, cols] -> packed codes [rows, cols/2] and scales e4m3 [rows, cols/16]."""
    rows, cols = y.shape
    blk = y.view(rows, cols // 16, 16)
    a = blk.abs().amax(dim=2)
    # tensors as divisors: torch turns a division by a number into a product with its reciprocal
    s = ((a / torch.full_like(a, 6.0)) * gs).clamp(max=448.0).to(torch.float8_e4m3fn)
    sv = s.float()
    r = torch.where(sv == 0, torch.zeros_like(sv), gs / sv)
    c = _e2m1_codes(blk * r[:, :, None]).view(rows, cols // 2, 2)
    return c[:, :, 0] + 16 * c[:, :, 1], s


def _mma_order(rows, cols, device):
    """Byte position of scale (row, 16-column block) in the tensor-core layout:
    512-byte atoms [rows/128][cols/64], byte (r % 32) * 16 + (r % 128) / 32 * 4 + j."""
    r = torch.arange(rows, device=device)[:, None]
    j = torch.arange(cols // 16, device=device)[None, :]
    return ((r // 128) * (cols // 64) + j // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4


def _to_mma(s, cols):
    rows = s.shape[0]
    out = torch.zeros((rows + 127) // 128 * 128 * (cols // 16), dtype=torch.uint8, device=s.device)
    out[_mma_order(rows, cols, s.device).reshape(-1)] = s.view(torch.uint8).reshape(-1)
    return out


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    g = _gen(seed)
    return {"norm": _prepare_norm, "gemv": _prepare_gemv, "balance": _prepare_balance}[case["op"]](case, g)


def _prepare_norm(case, g):
    T, H, quant = case["T"], case["H"], case["quant"]
    st = dict(case)
    # a block's output and a residual stream with some loud channels, as a trained model has
    st["x"] = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    loud = 1.0 + 19.0 * (torch.rand(H, generator=g, device=DEV) < 0.01)
    st["residual"] = (2.0 * torch.randn(T, H, generator=g, device=DEV) * loud).to(torch.bfloat16) if case["res"] else None
    st["weight"] = (1.0 + 0.1 * torch.randn(H, generator=g, device=DEV)).to(torch.bfloat16)
    # the global scale a warm-up fixed: 2688 over the largest value seen there
    st["gs"] = torch.full((1,), 2688.0 / 40.0, device=DEV) if quant == "nvfp4" else None
    st["y"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    st["residual_out"] = torch.empty_like(st["x"]) if case["res"] else None
    st["codes"] = st["scales"] = None
    if quant == "nvfp4":
        st["codes"] = torch.empty(T, H // 2, dtype=torch.uint8, device=DEV)
        rows = T if case["layout"] == "rows" else (T + 127) // 128 * 128
        st["scales"] = torch.zeros(rows * (H // 16), dtype=torch.uint8, device=DEV)
    elif quant == "e4m3":
        st["codes"] = torch.empty(T, H, dtype=torch.uint8, device=DEV)
        st["scales"] = torch.empty(T, (H + 127) // 128, dtype=torch.float32, device=DEV)
    return st


def _prepare_gemv(case, g):
    M, N, K = case["M"], case["N"], case["K"]
    st = dict(case)
    st["x"] = torch.randn(M, K, generator=g, device=DEV).to(torch.bfloat16)
    seg = [N] if case["segs"] == 1 else [max(32, N * 3 // 4 // 32 * 32), N]
    codes, scales, gss = [], [], []
    at = 0
    for i, end in enumerate(seg):          # one global scale per stacked projection
        w = (0.02 * (1 + i)) * torch.randn(end - at, K, generator=g, device=DEV)
        gs = 2688.0 / w.abs().amax()
        c, s = _nvfp4(w, gs)
        codes.append(c)
        scales.append(s.view(torch.uint8))
        gss.append(gs)
        at = end
        del w
    st["seg_end"] = seg
    st["b_codes"] = torch.cat(codes)
    st["b_scales"] = _to_mma(torch.cat(scales), K)
    st["b_gs"] = torch.stack(gss)
    st["out"] = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    return st


def _prepare_balance(case, g):
    T, E, k, S = case["T"], case["E"], case["k"], case["S"]
    st = dict(case)
    popular = 0.7 * torch.randn(E, generator=g, device=DEV)
    st["logits"] = torch.randn(T, E, generator=g, device=DEV) + popular
    ids = torch.topk(st["logits"], k, dim=1).indices.to(torch.int32)
    if case["pad"]:                         # padded tokens have no slot
        ids[torch.rand(T, generator=g, device=DEV) < 0.03] = -1
    st["ids"] = ids.contiguous()
    # ragged sequences, empty ones among them; a few tokens may stand behind the last
    cut = torch.randint(0, T + 1, (S + 1,), generator=g, device=DEV).sort().values
    cut[0] = 0
    cut[S] = max(1, T - T // 100)
    st["offsets"] = torch.cummax(cut.clamp(max=int(cut[S])), 0).values.to(torch.int32)
    st["counts"] = torch.empty(S, E, dtype=torch.int32, device=DEV)
    st["tokens"] = torch.empty(S, dtype=torch.int32, device=DEV)
    st["probs"] = torch.empty(S, E, dtype=torch.float32, device=DEV)
    st["loss"] = torch.empty(S, dtype=torch.float32, device=DEV)
    st["grad_loss"] = 1e-2 * (0.5 + torch.rand(S, generator=g, device=DEV))
    st["grad_weights"] = 1e-3 * torch.randn(T, k, generator=g, device=DEV)
    st["grad_logits"] = torch.empty(T, E, device=DEV)
    if case["do"] == "grad":                # what the loss's forward left
        c, n, _, _ = _loss_plain(st)
        st["counts"].copy_(c)
        st["tokens"].copy_(n)
    # scratch that a user's program keeps: 16 bytes per expert for each group of tokens, at most
    st["workspace"] = torch.empty(16 * (E + 32) * (1024 + S), dtype=torch.uint8, device=DEV)
    return st


# ---------------------------------------------------------------- plain forms
def _norm_plain(st):
    x, res = st["x"].float(), st["residual"]
    h = (x if res is None else x + res.float()).to(torch.bfloat16)
    hf = h.float()
    # the mean of squares in 64 bits, so that y does not depend on an order of summation
    rstd = (1.0 / torch.sqrt(hf.double().square().mean(dim=1, keepdim=True) + EPS)).float()
    yf = hf * rstd * st["weight"].float()
    y = yf.to(torch.bfloat16)
    out = {"y": y}
    if res is not None:
        out["residual"] = h
    if st["quant"] == "nvfp4":               # what the quantiser makes of y
        out["codes"], s = _nvfp4(y.float(), st["gs"])
        s8 = s.view(torch.uint8)
        out["scales"] = (_to_mma(s8, st["H"]) if st["layout"] == "mma" else s8.reshape(-1)).view(torch.float8_e4m3fn)
    elif st["quant"] == "e4m3":              # of the row before its rounding to bf16
        T, H = yf.shape
        grp = torch.nn.functional.pad(yf, (0, -H % 128)).view(T, -1, 128)
        a = grp.abs().amax(dim=2)
        top = torch.full_like(a, 448.0)
        r = torch.where(a == 0, torch.zeros_like(a), top / a)
        out["codes"] = (grp * r[:, :, None]).clamp(-448.0, 448.0).reshape(T, -1)[:, :H].to(torch.float8_e4m3fn)
        out["scales"] = a / top
    return out


def _gemv_plain(st):
    N, K = st["N"], st["K"]
    c = st["b_codes"]
    nib = torch.stack((c & 15, c >> 4), dim=2).view(N, K)
    lut = torch.tensor(E2M1 + [-v for v in E2M1], device=DEV)
    s = st["b_scales"][_mma_order(N, K, DEV)].view(torch.float8_e4m3fn).float()
    w = (lut[nib.int()].view(N, K // 16, 16) * s[:, :, None]).view(N, K)
    seg = torch.tensor(st["seg_end"], device=DEV)
    gs = st["b_gs"][torch.searchsorted(seg, torch.arange(N, device=DEV), right=True)]
    return ((st["x"].float() @ w.t()) / gs).to(torch.bfloat16)


def _rows_of(st):
    """Sequence of each token (S: none), and whether the token counts."""
    T, S = st["T"], st["S"]
    t = torch.arange(T, device=DEV, dtype=torch.int32)
    seq = torch.searchsorted(st["offsets"], t, right=True) - 1
    inside = (seq >= 0) & (seq < S)
    valid = inside & (st["ids"] >= 0).any(dim=1)
    return torch.where(valid, seq, torch.full_like(seq, S)), valid


def _probs_plain(st):
    l = st["logits"]
    if st["scoring"] == "softmax":
        e = torch.exp(l - l.amax(dim=1, keepdim=True))
        return e / e.sum(dim=1, keepdim=True), None
    s = 1.0 / (1.0 + torch.exp(-l))
    return s / s.sum(dim=1, keepdim=True), s


def _loss_plain(st):
    T, E, k, S = st["T"], st["E"], st["k"], st["S"]
    seq, valid = _rows_of(st)
    ids = st["ids"].long()
    flat = torch.where(ids >= 0, seq[:, None] * E + ids, torch.full_like(ids, S * E))
    counts = torch.zeros((S + 1) * E, dtype=torch.int64, device=DEV).scatter_add_(0, flat.reshape(-1), torch.ones_like(flat).reshape(-1))
    counts = counts[:S * E].view(S, E).to(torch.int32)
    n = torch.zeros(S + 1, dtype=torch.int64, device=DEV).scatter_add_(0, seq, torch.ones_like(seq))[:S]
    p, _ = _probs_plain(st)
    # long sums in 64 bits
    P = torch.zeros(S + 1, E, dtype=torch.float64, device=DEV).index_add_(0, seq, p.double())[:S]
    m = n.clamp(min=1).double()
    loss = (counts.double() * P).sum(dim=1) * (E / k) / (m * m)
    return counts, n.to(torch.int32), P.float(), loss.float()


def _grad_plain(st, counts, tokens):
    E, k = st["E"], st["k"]
    seq, valid = _rows_of(st)
    at = seq.clamp(max=st["S"] - 1)
    p, s = _probs_plain(st)
    n = tokens[at].float().clamp(min=1.0)
    coef = torch.where(valid, st["grad_loss"][at] * (E / k) / n / n, torch.zeros_like(n))
    c = counts[at].float()
    d = p * (c - (p * c).sum(dim=1, keepdim=True)) * coef[:, None]
    if s is not None:
        d = d * (1.0 - s)
    # the selected weights' part: softmax or normalised sigmoid over the row's slots
    ids = st["ids"].long()
    on = (ids >= 0) & valid[:, None]
    l = st["logits"].gather(1, ids.clamp(min=0))
    g = st["grad_weights"]
    if s is None:
        top = torch.where(on, l, torch.full_like(l, -1e30)).amax(dim=1, keepdim=True)
        v, slope = torch.where(on, torch.exp(l - top), torch.zeros_like(l)), torch.ones_like(l)
    else:
        sj = 1.0 / (1.0 + torch.exp(-l))
        v, slope = torch.where(on, sj, torch.zeros_like(l)), 1.0 - sj
    w = v / v.sum(dim=1, keepdim=True).clamp(min=1e-30)
    dj = w * (g - (g * w).sum(dim=1, keepdim=True)) * slope
    return d.scatter_add(1, ids.clamp(min=0), torch.where(on, dj, torch.zeros_like(dj)))


# ---------------------------------------------------------------- one pass
def run(st):
    if own:
        return _run_own(st)
    if st["op"] == "norm":
        return _norm_plain(st)
    if st["op"] == "gemv":
        return _gemv_plain(st)
    out = {}
    counts, tokens = st["counts"], st["tokens"]
    if st["do"] != "grad":
        counts, tokens, P, loss = _loss_plain(st)
        out = {"counts": counts, "tokens": tokens, "probs": P, "loss": loss}
    if st["do"] != "loss":
        out["grad_logits"] = _grad_plain(st, counts, tokens)
    return out


def _run_own(st):
    import nvfp4_moe_expert_topk_b200 as lib
    if st["op"] == "norm":
        quant = {"none": lib.NVFP4_QUANT_NONE, "nvfp4": lib.NVFP4_QUANT_NVFP4, "e4m3": lib.NVFP4_QUANT_E4M3}[st["quant"]]
        layout = lib.NVFP4_SCALES_MMA if st["layout"] == "mma" else lib.NVFP4_SCALES_ROWMAJOR
        lib.nvfp4_add_rmsnorm(st["x"], st["weight"], EPS, y=st["y"], residual=st["residual"], residual_out=st["residual_out"],
                              quant=quant, gs=st["gs"], codes=st["codes"], scales=st["scales"], scale_layout=layout)
        out = {"y": st["y"]}
        if st["res"]:
            out["residual"] = st["residual_out"]
        if st["quant"] == "nvfp4":
            out["codes"], out["scales"] = st["codes"], st["scales"].view(torch.float8_e4m3fn)
        elif st["quant"] == "e4m3":
            out["codes"], out["scales"] = st["codes"].view(torch.float8_e4m3fn), st["scales"]
        return out
    if st["op"] == "gemv":
        lib.nvfp4_gemv(st["x"], st["b_codes"], st["b_scales"], st["b_gs"], st["seg_end"], st["out"])
        return st["out"]
    scoring = lib.NVFP4_SCORING_SOFTMAX if st["scoring"] == "softmax" else lib.NVFP4_SCORING_SIGMOID
    out = {}
    if st["do"] != "grad":
        lib.nvfp4_moe_balance(st["logits"], st["ids"], st["k"], st["counts"], st["tokens"], st["probs"], st["loss"],
                              st["workspace"], seq_offsets=st["offsets"], scoring=scoring)
        out = {"counts": st["counts"], "tokens": st["tokens"], "probs": st["probs"], "loss": st["loss"]}
    if st["do"] != "loss":
        lib.nvfp4_moe_balance_backward(st["logits"], st["ids"], st["k"], st["counts"], st["tokens"], st["grad_loss"],
                                       st["grad_logits"], grad_weights=st["grad_weights"], seq_offsets=st["offsets"],
                                       scoring=scoring)
        out["grad_logits"] = st["grad_logits"]
    return out


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _norm_exact, "gemv": _gemv_exact, "balance": _balance_exact}[case["op"]](st)


def _norm_exact(st):
    h = st["x"].double()
    if st["residual"] is not None:
        h = (h + st["residual"].double()).to(torch.bfloat16).double()
    y = h / (h.pow(2).sum(dim=1, keepdim=True) / st["H"] + EPS).sqrt() * st["weight"].double()
    out = {"y": y}
    if st["residual"] is not None:
        out["residual"] = h
    T, H = y.shape
    if st["quant"] == "nvfp4":
        q = y.to(torch.bfloat16).double()            # the NVFP4 rows are those of the rounded y
        # the packed codes are whole numbers, one per value: they have no value in 64 bits of their own
        v = q.view(T, H // 16, 16).abs().amax(dim=2) * st["gs"].double() / 6.0
        e = torch.floor(torch.log2(v.clamp(min=2.0 ** -6)))
        step = torch.pow(2.0, e - 3)                 # spacing of the 8-bit scales around v
        s = (torch.round(v / step) * step).clamp(max=448.0)
        if st["layout"] == "mma":
            full = torch.zeros((T + 127) // 128 * 128, H // 16, dtype=torch.float64, device=DEV)
            full[:T] = s
            s = full.view(-1, 4, 32, H // 64, 4).permute(0, 3, 2, 1, 4)
        out["codes"], out["scales"] = None, s.reshape(-1)
    elif st["quant"] == "e4m3":
        pad = torch.zeros(T, (H + 127) // 128 * 128, dtype=torch.float64, device=DEV)
        pad[:, :H] = y
        a = pad.view(T, -1, 128).abs().amax(dim=2)
        v = pad.view(T, -1, 128) / torch.where(a > 0, a, torch.ones_like(a))[:, :, None] * 448.0
        step = torch.pow(2.0, torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        out["codes"], out["scales"] = (torch.round(v / step) * step).reshape(T, -1)[:, :H], a / 448.0
    return out


def _gemv_exact(st):
    M, N, K = st["M"], st["N"], st["K"]
    x = st["x"].double()
    out = torch.empty(M, N, dtype=torch.float64, device=DEV)
    blocks = (N + 127) // 128
    sc = st["b_scales"].view(blocks, K // 64, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(blocks * 128, K // 16)
    ends = [0] + list(st["seg_end"])
    for i in range(len(ends) - 1):
        for a in range(ends[i], ends[i + 1], 8192):
            b = min(a + 8192, ends[i + 1])
            byte = st["b_codes"][a:b].to(torch.int32)
            nib = torch.stack((byte % 16, byte // 16), dim=2).view(b - a, K)
            mag = (nib % 8).double()                 # 0 0.5 1 1.5 | 2 3 | 4 6
            mag = torch.where(mag < 4, mag / 2, torch.where(mag < 6, mag - 2, 2 * mag - 8))
            val = torch.where(nib >= 8, -mag, mag)
            byte = sc[a:b].to(torch.int32)
            ex, fr = byte // 8, (byte % 8).double()
            s = torch.where(ex == 0, fr / 512.0, (1 + fr / 8) * torch.pow(2.0, (ex - 7).double()))
            w = val.view(b - a, K // 16, 16) * s[:, :, None] / st["b_gs"][i].double()
            out[:, a:b] = x @ w.view(b - a, K).t()
    return out


def _balance_exact(st):
    T, E, k, S = st["T"], st["E"], st["k"], st["S"]
    l = st["logits"].double()
    score = torch.sigmoid(l) if st["scoring"] == "sigmoid" else torch.exp(l - l.logsumexp(dim=1, keepdim=True))
    total = score.sum(dim=1, keepdim=True)
    p = score / total
    ids = st["ids"].long()
    off = [int(v) for v in st["offsets"].tolist()]
    counts = torch.zeros(S, E, dtype=torch.float64, device=DEV)
    tokens = torch.zeros(S, dtype=torch.float64, device=DEV)
    P = torch.zeros(S, E, dtype=torch.float64, device=DEV)
    grad = torch.zeros(T, E, dtype=torch.float64, device=DEV)
    loss = torch.zeros(S, dtype=torch.float64, device=DEV)
    for s in range(S):
        a, b = off[s], off[s + 1]
        live = (ids[a:b] >= 0).any(dim=1)
        n = int(live.sum())
        if n == 0:
            continue
        row = ids[a:b][live]
        f = torch.bincount(row[row >= 0], minlength=E).double()
        pr = p[a:b][live]
        counts[s], tokens[s], P[s] = f, n, pr.sum(dim=0)
        c = E / (k * float(n) ** 2)
        loss[s] = c * (f * P[s]).sum()
        # d loss / d p = c f; through p = score / total, then through the score
        d = c * st["grad_loss"][s].double() * (f - pr @ f[:, None])
        sl = score[a:b][live]
        grad_row = d * pr * (1 - sl) if st["scoring"] == "sigmoid" else d * pr
        # the selected weights: w = v / sum v over the slots
        pick = sl.gather(1, row.clamp(min=0)) * (row >= 0)
        w = pick / pick.sum(dim=1, keepdim=True)
        gw = st["grad_weights"][a:b][live].double()
        dw = w * (gw - (gw * w).sum(dim=1, keepdim=True))
        if st["scoring"] == "sigmoid":
            dw = dw * (1 - sl.gather(1, row.clamp(min=0)))
        grad_row.scatter_add_(1, row.clamp(min=0), dw * (row >= 0))
        at = torch.arange(a, b, device=DEV)[live]
        grad[at] = grad_row
    out = {}
    if st["do"] != "grad":
        out = {"counts": counts.to(torch.int32), "tokens": tokens.to(torch.int32), "probs": P, "loss": loss}
    if st["do"] != "loss":
        out["grad_logits"] = grad
    return out
