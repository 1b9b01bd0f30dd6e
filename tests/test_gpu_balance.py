"""nvfp4_moe_balance and its backward against their formulas in 64 bits.

Tolerances, derived from the arithmetic (u = 2^-24):
 - a score (exp or sigmoid) is off by at most 4 u plus, for softmax, the
   rounding of its argument (u * max|l - max l|, of the exponent: relative);
   the sum of E positive scores by E / 32 + 8 additions; reciprocal and product
   2 u: rel(p) <= (E / 32 + 16 + spread) u with spread = 2 max|l - max l|
   (sigmoid: 2 max|l|, the same argument);
 - P adds at most chunk / 8 + 8 of them in fp32, then in 64 bits; all terms
   are positive, so rel(P) <= rel(p) + (chunk / 8 + 10) u, loss alike + 2 u;
 - a gradient entry is p * (c - sum p c) * coef: its error is at most
   coef * p * (|c| + sum p c) * (2 rel(p) + (E / 32 + 16) u), for sigmoid the
   factor 1 - s adds u / (1 - s) * (1 - s) <= 4 u of the same size; the weights'
   part |w| (|g| + sum |g| w) * (rel(w) + 16 u) with rel(w) <= (40 + spread) u."""
import numpy as np
import pytest
import torch

import oracle as O
from nvfp4_moe_expert_topk_b200 import (NVFP4_SCORING_SIGMOID, NVFP4_SCORING_SOFTMAX, Nvfp4Error, nvfp4_moe_balance,
                                        nvfp4_moe_balance_backward, nvfp4_moe_balance_workspace_size, nvfp4_moe_topk,
                                        nvfp4_moe_topk_shared)

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
SCORING = {"softmax": NVFP4_SCORING_SOFTMAX, "sigmoid": NVFP4_SCORING_SIGMOID}


def chunk_bound(T):
    """No chunk is longer than this (the chunks are a share of the batch)."""
    return T / 128 + 64


def scores64(l, scoring):
    l = l.astype(np.float64)
    if scoring == "softmax":
        with np.errstate(invalid="ignore"):
            m = l.max(axis=1, keepdims=True)
            s = np.exp(l - np.where(np.isfinite(m), m, 0))
    else:
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-l))
    tot = s.sum(axis=1, keepdims=True)
    return s, np.where(tot > 0, s / np.where(tot > 0, tot, 1), 0.0)


def loss64(l, ids, k, off, scoring):
    """counts, tokens, P, loss per sequence."""
    E, S = l.shape[1], len(off) - 1
    ids = ids[:, :k]
    ok = (ids >= 0) & (ids < E)
    live = ok.any(axis=1)
    p = np.zeros(l.shape)
    p[live] = scores64(l[live], scoring)[1]
    counts, tokens = np.zeros((S, E), np.int64), np.zeros(S, np.int64)
    P, loss = np.zeros((S, E)), np.zeros(S)
    for s in range(S):
        sl = slice(off[s], off[s + 1])
        counts[s] = np.bincount(ids[sl][ok[sl]], minlength=E)
        tokens[s] = live[sl].sum()
        P[s] = p[sl].sum(axis=0)
        if tokens[s]:
            loss[s] = E / (k * float(tokens[s]) ** 2) * (counts[s] * P[s]).sum()
    return counts, tokens, P, loss


def weights64(l, ids, k, scoring):
    """Renormalised weights over the row's slots (0 in skipped ones), their slope."""
    ids = ids[:, :k]
    ok = (ids >= 0) & (ids < l.shape[1])
    sel = np.take_along_axis(l.astype(np.float64), np.clip(ids, 0, l.shape[1] - 1), axis=1)
    if scoring == "softmax":
        m = np.where(ok, sel, -np.inf).max(axis=1, keepdims=True)
        v, slope = np.where(ok, np.exp(sel - np.where(np.isfinite(m), m, 0)), 0.0), np.ones(sel.shape)
    else:
        with np.errstate(over="ignore"):
            sg = 1.0 / (1.0 + np.exp(-sel))
        v, slope = np.where(ok, sg, 0.0), 1.0 - sg
    tot = v.sum(axis=1, keepdims=True)
    return np.where(tot > 0, v / np.where(tot > 0, tot, 1), 0.0), slope, ok


def grad64(l, ids, k, off, scoring, gl, gw):
    """(gradient, bound of its error in units of u)."""
    T, E = l.shape
    counts, tokens, _, _ = loss64(l, ids, k, off, scoring)
    fin = np.where(np.isfinite(l), l, 0)
    spread = 2 * (np.abs(fin).max() if scoring == "sigmoid" else (fin.max(axis=1) - fin.min(axis=1)).max())
    relp = E / 32 + 16 + spread
    grad, err = np.zeros((T, E)), np.zeros((T, E))
    for s in range(len(off) - 1):
        if not tokens[s]:
            continue
        t = np.arange(off[s], off[s + 1])
        okrow = ((ids[t, :k] >= 0) & (ids[t, :k] < E)).any(axis=1)
        t = t[okrow]
        sc, p = scores64(l[t], scoring)
        c = counts[s].astype(np.float64)[None]
        coef = float(gl[s]) * E / (k * float(tokens[s]) ** 2)
        dot = (p * c).sum(axis=1, keepdims=True)
        grad[t] = coef * p * (c - dot)
        err[t] = abs(coef) * p * (c + dot) * (2 * relp + E / 32 + 20)
        if scoring == "sigmoid":
            grad[t] *= 1 - sc
        if gw is not None:
            w, slope, ok = weights64(l[t], ids[t], k, scoring)
            g = np.where(ok, gw[t].astype(np.float64), 0)
            d = w * (g - (g * w).sum(axis=1, keepdims=True)) * slope
            e = w * (np.abs(g) + (np.abs(g) * w).sum(axis=1, keepdims=True)) * (56 + spread)
            for j in range(k):
                at = np.clip(ids[t, j], 0, E - 1)
                np.add.at(grad, (t, at), np.where(ok[:, j], d[:, j], 0))
                np.add.at(err, (t, at), np.where(ok[:, j], e[:, j], 0))
    return grad, err


class Case:
    def __init__(self, T, E, k, S=1, scoring="softmax", seed=0, pad=0.0, extra=0, spread=1.5, off=None, skip=0.0):
        rng = np.random.default_rng(seed)
        self.T, self.E, self.k, self.scoring = T, E, k, scoring
        self.l = rng.normal(0, spread, (T, E)).astype(np.float32)
        self.ids = np.argsort(-self.l, axis=1, kind="stable")[:, :k].astype(np.int32)
        if extra:                                   # shared-expert slots behind the routed ones
            self.ids = np.concatenate([self.ids, np.tile(np.arange(E, E + extra, dtype=np.int32), (T, 1))], axis=1)
        self.ids = np.ascontiguousarray(self.ids)
        if skip:
            self.ids[:, :k][rng.random((T, k)) < skip] = -1
        if pad:
            self.ids[rng.random(T) < pad, :k] = -1
        if off is None and S > 0:
            cut = np.sort(rng.integers(0, T + 1, S + 1))
            cut[0], cut[-1] = 0, max(cut[-1], T - T // 50)
            off = cut
        self.off = np.array([0, T] if off is None else off, np.int64)
        self.plain = off is None                    # no offsets passed
        self.S = len(self.off) - 1
        self.gl = rng.uniform(-2, 2, self.S).astype(np.float32)
        self.gw = rng.normal(0, 1, (T, k)).astype(np.float32)

    def dev(self):
        o = None if self.plain else torch.from_numpy(self.off.astype(np.int32)).to(DEV)
        return torch.from_numpy(self.l).to(DEV), torch.from_numpy(self.ids).to(DEV), o

    def forward(self, stream=None, ws=None):
        l, ids, o = self.dev()
        S, E = self.S, self.E
        out = [torch.full((S, E), -9, dtype=torch.int32, device=DEV), torch.full((S,), -9, dtype=torch.int32, device=DEV),
               torch.full((S, E), float("nan"), device=DEV), torch.full((S,), float("nan"), device=DEV)]
        need = nvfp4_moe_balance_workspace_size(self.T, S, E)
        guarded = ws is None
        if guarded:
            ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device=DEV)   # any contents: NaN here
        nvfp4_moe_balance(l, ids, self.k, *out, ws[:need], seq_offsets=o, scoring=SCORING[self.scoring], stream=stream)
        torch.cuda.synchronize()
        assert not guarded or (ws[need:] == 0xFF).all()
        return out

    def backward(self, gw=True):
        l, ids, o = self.dev()
        counts, tokens, _, _ = loss64(self.l, self.ids, self.k, self.off, self.scoring)
        guard = torch.full((self.T + 1, self.E), 5.0, device=DEV)
        nvfp4_moe_balance_backward(l, ids, self.k, torch.from_numpy(counts.astype(np.int32)).to(DEV),
                                   torch.from_numpy(tokens.astype(np.int32)).to(DEV), torch.from_numpy(self.gl).to(DEV),
                                   guard[:self.T], torch.from_numpy(self.gw).to(DEV) if gw else None, seq_offsets=o,
                                   scoring=SCORING[self.scoring])
        torch.cuda.synchronize()
        assert (guard[self.T] == 5.0).all()
        return guard[:self.T].cpu().numpy()

    def check(self):
        counts, tokens, P, loss = (t.cpu().numpy() for t in self.forward())
        wc, wt, wP, wl = loss64(self.l, self.ids, self.k, self.off, self.scoring)
        np.testing.assert_array_equal(counts, wc)
        np.testing.assert_array_equal(tokens, wt)
        fin = np.where(np.isfinite(self.l), self.l, 0)
        if self.T:
            spread = 2 * (np.abs(fin).max() if self.scoring == "sigmoid" else (fin.max(axis=1) - fin.min(axis=1)).max())
        else:
            spread = 0
        rel = (self.E / 32 + 16 + spread + chunk_bound(self.T) / 8 + 12) * U
        np.testing.assert_allclose(P, wP, rtol=rel, atol=1e-37)
        np.testing.assert_allclose(loss, wl, rtol=rel + 2 * U, atol=1e-37)
        for gw in (True, False):
            got = self.backward(gw)
            want, err = grad64(self.l, self.ids, self.k, self.off, self.scoring, self.gl, self.gw if gw else None)
            bad = np.abs(got - want) > err * U + 1e-37
            assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], (err * U)[bad][:4])
        return counts, tokens, P, loss


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 5, 5), (7, 33, 4), (64, 48, 6), (100, 127, 3), (65, 128, 8),
                                   (50, 130, 6), (200, 256, 8), (513, 384, 6), (31, 500, 10), (40, 513, 6), (33, 1000, 32),
                                   (20, 1023, 7), (70, 1024, 32)])
def test_sizes(T, E, k, scoring):
    Case(T, E, k, S=0, scoring=scoring, seed=T + E).check()
    Case(T, E, k, S=3, scoring=scoring, seed=T + E, pad=0.2).check()


@pytest.mark.parametrize("T,E,k", [(t, E, k) for E, k in [(1, 1), (7, 3), (48, 6), (130, 6), (384, 6), (509, 8), (1024, 5)]
                                   for t in (128 * 1212 // (E + 700), 128 * 1212 // (E + 700) + 1, 600, 1537, 2049)])
def test_borders_between_forms(T, E, k):
    """Batch lengths around those where the number of launches and the tokens
    per chunk change; more sequences than tokens in one of them."""
    for S, scoring in ((0, "softmax"), (2, "sigmoid"), (13, "softmax"), (700, "sigmoid")):
        Case(T, E, k, S=S, scoring=scoring, seed=T + S, pad=0.1).check()


@pytest.mark.parametrize("T,E", [(5000, 40), (5000, 513), (20000, 1022)])
def test_sums_over_chunks_add_up(T, E):
    """Logits of 0: every token adds 1 / E to every probability sum and the
    counts are known, so the sums over chunks and their borders are seen
    whole, for one sequence and for many of odd lengths."""
    l = torch.zeros(T, E, device=DEV)
    ids = (torch.arange(T, device=DEV)[:, None] * 3 + torch.arange(2, device=DEV)).remainder(E).to(torch.int32)
    for S in (1, 7, 160):
        off = (torch.arange(S + 1, dtype=torch.int64) * T // S).to(torch.int32)
        counts, tokens = (torch.empty(*n, dtype=torch.int32, device=DEV) for n in ((S, E), (S,)))
        probs, loss = torch.empty(S, E, device=DEV), torch.empty(S, device=DEV)
        ws = torch.full((nvfp4_moe_balance_workspace_size(T, S, E),), 0xFF, dtype=torch.uint8, device=DEV)
        nvfp4_moe_balance(l, ids, 2, counts, tokens, probs, loss, ws, seq_offsets=off.to(DEV))
        n = off.diff()
        assert torch.equal(tokens.cpu(), n)
        host = ids.cpu()
        want = torch.stack([torch.bincount(host[a:b].flatten(), minlength=E) for a, b in zip(off[:-1], off[1:])])
        assert torch.equal(counts.cpu(), want.to(torch.int32))
        # 1 / E rounded, then fp32 sums of at most T / 64 terms by a warp and of 16 warps, and the last rounding
        bound = (T / 64 + 20) * 2.0 ** -24
        P = n[:, None].double() / E
        assert ((probs.cpu().double() - P).abs() <= bound * P).all()
        assert ((loss.cpu().double() - 1).abs() <= 2 * bound).all()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_long_batch(scoring):
    Case(20011, 384, 6, S=0, scoring=scoring, seed=3).check()
    Case(30000, 64, 4, S=17, scoring=scoring, seed=4, pad=0.05).check()


@pytest.mark.parametrize("off", [[0, 0], [0, 0, 0, 40], [0, 40, 40, 40], [0, 1, 2, 3, 4], [5, 9, 30], [0, 8, 16, 24, 32, 40],
                                 [0, 7, 8, 9, 39], [40, 40], [3, 3, 3]])
def test_offsets(off):
    """Empty sequences, one token each, edges on and off the chunk borders,
    tokens before the first and behind the last sequence."""
    c = Case(40, 24, 3, off=off, seed=len(off))
    c.check()
    got = c.backward()
    outside = [t for t in range(40) if t < off[0] or t >= off[-1]]
    assert (got[outside] == 0).all()


def test_many_sequences():
    off = np.sort(np.random.default_rng(1).integers(0, 3001, 701))
    Case(3000, 40, 4, off=off, seed=2, scoring="sigmoid").check()
    Case(37, 16, 2, S=200, seed=3).check()             # more sequences than tokens


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_padding_rows_are_not_read(scoring):
    """A token without a slot counts nowhere, whatever its logits hold."""
    c = Case(90, 72, 4, S=4, scoring=scoring, seed=5, pad=0.3)
    pad = (c.ids < 0).all(axis=1)
    assert pad.any() and not pad.all()
    a = [t.cpu().numpy() for t in c.forward()] + [c.backward()]
    c.l[pad] = np.nan
    c.l[np.flatnonzero(pad)[0]] = np.inf
    b = [t.cpu().numpy() for t in c.forward()] + [c.backward()]
    for x, y in zip(a, b):
        np.testing.assert_array_equal(x, y)
    assert (b[-1][pad] == 0).all()
    c = Case(30, 72, 4, S=2, scoring=scoring, seed=5, pad=1.0)      # nothing but padding
    counts, tokens, P, loss = (t.cpu().numpy() for t in c.forward())
    assert not counts.any() and not tokens.any() and not P.any() and not loss.any() and not c.backward().any()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_skipped_and_out_of_range_slots(scoring):
    c = Case(120, 40, 5, S=3, scoring=scoring, seed=6, skip=0.3)
    c.ids[3, 1], c.ids[9, 0] = 40, 2 ** 31 - 1           # out of range: skipped slots
    c.check()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_one_expert_twice(scoring):
    """Slots of a row that name the same expert count and add up each."""
    c = Case(60, 20, 4, S=2, scoring=scoring, seed=7)
    c.ids[::3, 1] = c.ids[::3, 0]
    c.ids[1::3, :] = c.ids[1::3, :1]
    c.check()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_masked_logits(scoring):
    """-inf and the lowest fp32 value: no probability, no gradient; a row of
    nothing else has no probability at all."""
    c = Case(50, 36, 3, S=2, scoring=scoring, seed=8)
    rng = np.random.default_rng(8)
    m = rng.random(c.l.shape) < 0.4
    m[np.arange(50)[:, None], c.ids] = False
    c.l[m] = -np.inf
    c.l[4] = -np.inf
    counts, tokens, P, loss = c.check()
    assert np.isfinite(P).all()
    low = c.l.copy()
    c.l[m] = np.finfo(np.float32).min
    got = c.backward()
    assert np.isfinite(got).all()
    want, err = grad64(low, c.ids, c.k, c.off, scoring, c.gl, c.gw)
    if scoring == "sigmoid":                             # 1 / (1 + exp(3e38)) = 0 as well
        assert (np.abs(got - want) <= err * U + 1e-37).all()
    else:
        # row 4 holds the lowest value and -inf only: a softmax over its places of the lowest value
        zero = m.copy()
        zero[4] = False
        assert (got[zero] == 0).all()
        assert (got[4][c.l[4] == -np.inf] == 0).all()


def test_extreme_logits():
    """Logits far apart and far from zero (softmax is shifted by the maximum;
    a sigmoid's arguments stay where fp32 holds it)."""
    c = Case(40, 64, 4, S=2, seed=9, spread=30.0)
    c.l += 1000.0
    c.l[0] -= 5000.0
    c.check()
    Case(40, 64, 4, S=2, seed=9, spread=12.0, scoring="sigmoid").check()


def test_shared_slots_are_not_counted():
    """The rows of nvfp4_moe_topk_shared: k routed slots, then the shared ones."""
    Case(77, 48, 6, S=2, seed=10, extra=2).check()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_unaligned_logits(scoring):
    """Rows that do not start on 16 bytes (a view into a larger buffer)."""
    c = Case(64, 48, 4, S=0, scoring=scoring, seed=11)
    want, err = grad64(c.l, c.ids, c.k, c.off, scoring, c.gl, c.gw)
    a = [t.cpu().numpy() for t in c.forward()]
    for shift in (1, 2, 3):
        buf = torch.zeros(64 * 48 + 4, device=DEV)
        l = buf[shift:shift + 64 * 48].view(64, 48)
        l.copy_(torch.from_numpy(c.l))
        ids = torch.from_numpy(c.ids).to(DEV)
        out = [torch.empty(1, 48, dtype=torch.int32, device=DEV), torch.empty(1, dtype=torch.int32, device=DEV),
               torch.empty(1, 48, device=DEV), torch.empty(1, device=DEV)]
        ws = torch.empty(nvfp4_moe_balance_workspace_size(64, 1, 48), dtype=torch.uint8, device=DEV)
        nvfp4_moe_balance(l, ids, 4, *out, ws, scoring=SCORING[scoring])
        gbuf = torch.full((64 * 48 + 4,), 8.0, device=DEV)
        g = gbuf[shift:shift + 64 * 48].view(64, 48)
        nvfp4_moe_balance_backward(l, ids, 4, out[0], out[1], torch.from_numpy(c.gl).to(DEV), g,
                                   torch.from_numpy(c.gw).to(DEV), scoring=SCORING[scoring])
        np.testing.assert_array_equal(out[0].cpu().numpy(), a[0])
        np.testing.assert_allclose(out[2].cpu().numpy(), a[2], rtol=100 * U)
        assert (np.abs(g.cpu().numpy() - want) <= err * U + 1e-37).all()
        assert (gbuf[:shift] == 8.0).all() and (gbuf[shift + 64 * 48:] == 8.0).all()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_gradient_against_differences(scoring):
    """The kernel's gradient against central differences of the 64-bit loss
    (step 1e-4: the differences are off by its square and by 1e-12 / step)."""
    c = Case(24, 12, 3, S=2, scoring=scoring, seed=12, pad=0.1)
    got = c.backward()

    def total(l):
        _, _, _, loss = loss64(l, c.ids, c.k, c.off, scoring)
        w, _, ok = weights64(l, c.ids, c.k, scoring)
        inside = np.zeros(c.T, bool)
        inside[c.off[0]:c.off[-1]] = True
        return (loss * c.gl).sum() + (w * c.gw * ok)[inside].sum()

    l0 = c.l.astype(np.float64)
    want = np.zeros_like(l0)
    h = 1e-4
    for t in range(c.T):
        for e in range(c.E):
            l = l0.copy()
            l[t, e] += h
            up = total(l)
            l[t, e] -= 2 * h
            want[t, e] = (up - total(l)) / (2 * h)
    np.testing.assert_allclose(got, want, rtol=1e-5, atol=5e-7)


def test_perfect_balance_has_loss_one_and_no_gradient():
    E, k, T = 16, 4, 64
    c = Case(T, E, k, S=0, seed=1)
    c.l[:] = 0.25
    c.ids = ((np.arange(T)[:, None] * k + np.arange(k)[None]) % E).astype(np.int32)
    counts, tokens, P, loss = c.check()
    assert (counts == T * k // E).all() and abs(loss[0] - 1.0) < 1e-6
    assert np.abs(c.backward(gw=False)).max() < 1e-6


def test_empty_batch():
    c = Case(0, 8, 2, off=[0, 0, 0], seed=0)
    counts, tokens, P, loss = (t.cpu().numpy() for t in c.forward())
    assert not counts.any() and not tokens.any() and not P.any() and not loss.any()
    c.backward()


def test_same_bits_every_time():
    """No result depends on timing: repeated calls, a smaller call in between
    on the same workspace, a side stream, a replayed graph."""
    c = Case(9000, 384, 6, S=5, seed=13, pad=0.02)
    ws = torch.empty(nvfp4_moe_balance_workspace_size(c.T, c.S, c.E), dtype=torch.uint8, device=DEV)
    first = c.forward(ws=ws)
    g1 = c.backward()
    small = Case(50, 384, 6, S=2, seed=14)
    small.forward(ws=ws)
    for _ in range(3):
        for a, b in zip(first, c.forward(ws=ws)):
            assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    l, ids, o = c.dev()
    torch.cuda.synchronize()
    out = [torch.empty_like(t) for t in first]
    nvfp4_moe_balance(l, ids, c.k, *out, ws, seq_offsets=o, stream=side)
    side.synchronize()
    for a, b in zip(first, out):
        assert torch.equal(a, b)
    np.testing.assert_array_equal(g1, c.backward())
    grad = torch.empty(c.T, c.E, device=DEV)
    gl, gw = torch.from_numpy(c.gl).to(DEV), torch.from_numpy(c.gw).to(DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nvfp4_moe_balance(l, ids, c.k, *out, ws, seq_offsets=o)
        nvfp4_moe_balance_backward(l, ids, c.k, out[0], out[1], gl, grad, gw, seq_offsets=o)
    for t in out:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, out):
        assert torch.equal(a, b)
    np.testing.assert_array_equal(grad.cpu().numpy(), g1)


@pytest.mark.parametrize("seed", range(16))
def test_random_shapes(seed):
    rng = np.random.default_rng(700 + seed)
    E = int(rng.integers(1, 1025))
    Case(int(np.exp(rng.uniform(0, 7.5))), E, int(rng.integers(1, min(32, E) + 1)), S=int(rng.integers(0, 20)),
         scoring=str(rng.choice(["softmax", "sigmoid"])), seed=seed, pad=float(rng.choice([0, 0.3])),
         skip=float(rng.choice([0, 0.2])), spread=float(rng.choice([0.5, 4.0]))).check()


def test_after_the_router():
    """nvfp4_moe_topk -> balance -> backward, as a training step makes them."""
    rng = np.random.default_rng(3)
    l = torch.from_numpy(rng.normal(0, 1, (700, 96)).astype(np.float32)).to(DEV)
    for shared in (0, 1):
        ids = torch.empty(700, 6 + shared, dtype=torch.int32, device=DEV)
        w = torch.empty(700, 6 + shared, device=DEV)
        if shared:
            nvfp4_moe_topk_shared(l, 6, shared, ids, w, NVFP4_SCORING_SIGMOID)
        else:
            nvfp4_moe_topk(l, 6, ids, w, NVFP4_SCORING_SIGMOID)
        c = Case(700, 96, 6, S=0, scoring="sigmoid")
        c.l, c.ids = l.cpu().numpy(), ids.cpu().numpy()
        np.testing.assert_array_equal(c.ids[:, :6], O.topk(c.l, 6, "sigmoid")[0])
        counts, tokens, P, loss = c.check()
        assert tokens[0] == 700 and counts.sum() == 4200


def test_refusals():
    l = torch.zeros(10, 8, device=DEV)
    ids = torch.zeros(10, 2, dtype=torch.int32, device=DEV)
    ok = dict(logits=l, topk_ids=ids, k=2, counts=torch.zeros(1, 8, dtype=torch.int32, device=DEV),
              tokens=torch.zeros(1, dtype=torch.int32, device=DEV), probs=torch.zeros(1, 8, device=DEV),
              loss=torch.zeros(1, device=DEV), workspace=torch.zeros(1 << 16, dtype=torch.uint8, device=DEV))
    nvfp4_moe_balance(**ok)
    for change, match in [(dict(logits=l.half()), "logits must be"), (dict(topk_ids=ids.long()), "topk_ids must be"),
                          (dict(topk_ids=ids[:9]), "topk_ids must be"), (dict(k=3), "topk_ids must be"),
                          (dict(counts=ids), "counts must hold"), (dict(tokens=ids[:, 0].contiguous()), "tokens must hold"),
                          (dict(loss=None), "loss is required"), (dict(probs=l), "probs must hold"),
                          (dict(logits=l.t()), "logits must be contiguous"), (dict(workspace=ids), "workspace must be"),
                          (dict(seq_offsets=torch.zeros(3, dtype=torch.int32, device=DEV)), "must hold"),
                          (dict(seq_offsets=torch.zeros(2, dtype=torch.int64, device=DEV)), "seq_offsets must be"),
                          (dict(seq_offsets=torch.zeros(2, dtype=torch.int32)), "CUDA tensor")]:
        with pytest.raises(ValueError, match=match):
            nvfp4_moe_balance(**dict(ok, **change))
    with pytest.raises(Nvfp4Error) as e:
        nvfp4_moe_balance(**dict(ok, workspace=ok["workspace"][:16]))
    assert e.value.status == -4
    with pytest.raises(Nvfp4Error) as e:
        nvfp4_moe_balance(**dict(ok, scoring=5))
    assert e.value.status == -1
    back = dict(logits=l, topk_ids=ids, k=2, counts=ok["counts"], tokens=ok["tokens"], grad_loss=ok["loss"],
                grad_logits=torch.zeros(10, 8, device=DEV))
    nvfp4_moe_balance_backward(**back)
    for change, match in [(dict(grad_logits=l[:9]), "grad_logits must hold"), (dict(grad_loss=l), "grad_loss must hold"),
                          (dict(grad_weights=l), "grad_weights must hold"), (dict(grad_weights=ids), "grad_weights must be")]:
        with pytest.raises(ValueError, match=match):
            nvfp4_moe_balance_backward(**dict(back, **change))


def sigmoid_grad64(c, gw):
    """(gradient, bound) of the sigmoid form where sigmoids are close to 1: the
    slope 1 - sigmoid(l) is taken as sigmoid(-l) on both sides, and every bound
    carries it.  As above, with rel(slope) <= (2 max|l| + 10) u on top."""
    T, E = c.l.shape
    counts, tokens, _, _ = loss64(c.l, c.ids, c.k, c.off, "sigmoid")
    spread = 2 * np.abs(np.where(np.isfinite(c.l), c.l, 0)).max()
    relp = E / 32 + 16 + spread
    grad, err = np.zeros((T, E)), np.zeros((T, E))
    for s in range(c.S):
        t = np.arange(c.off[s], c.off[s + 1])
        t = t[((c.ids[t, :c.k] >= 0) & (c.ids[t, :c.k] < E)).any(axis=1)]
        if not len(t):
            continue
        l = c.l[t].astype(np.float64)
        p = scores64(c.l[t], "sigmoid")[1]
        with np.errstate(over="ignore"):
            slope = 1.0 / (1.0 + np.exp(l))
        n = counts[s].astype(np.float64)[None]
        coef = float(c.gl[s]) * E / (c.k * float(tokens[s]) ** 2)
        dot = (p * n).sum(axis=1, keepdims=True)
        grad[t] = coef * p * (n - dot) * slope
        err[t] = abs(coef) * p * (n + dot) * slope * (2 * relp + E / 32 + 30 + spread)
        if gw:
            w, _, ok = weights64(c.l[t], c.ids[t], c.k, "sigmoid")
            at = np.clip(c.ids[t, :c.k], 0, E - 1)
            own = np.take_along_axis(slope, at, axis=1)
            g = np.where(ok, c.gw[t].astype(np.float64), 0)
            d = w * (g - (g * w).sum(axis=1, keepdims=True)) * own
            e = w * (np.abs(g) + (np.abs(g) * w).sum(axis=1, keepdims=True)) * own * (66 + 2 * spread)
            for j in range(c.k):
                np.add.at(grad, (t, at[:, j]), np.where(ok[:, j], d[:, j], 0))
                np.add.at(err, (t, at[:, j]), np.where(ok[:, j], e[:, j], 0))
    return grad, err


@pytest.mark.parametrize("lo,hi", [(8, 14), (14, 30), (-30, 30), (40, 80), (-5, 16)])
@pytest.mark.parametrize("T,E,k", [(40, 64, 4), (33, 130, 6), (300, 384, 6), (21, 1023, 7)])
def test_saturated_sigmoids_keep_their_slope(T, E, k, lo, hi):
    """Gradients of experts whose sigmoid is 1 in fp32: their slope e^-l is
    far from 0, and the gradient has it to fp32 accuracy."""
    c = Case(T, E, k, S=2, scoring="sigmoid", seed=E + hi, pad=0.1)
    c.l = np.random.default_rng(hi).uniform(lo, hi, (T, E)).astype(np.float32)
    for gw in (True, False):
        got = c.backward(gw)
        want, err = sigmoid_grad64(c, gw)
        assert (want != 0).any()
        bad = np.abs(got - want) > err * U + 1e-37
        assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], (err * U)[bad][:4])


def check_low(c):
    """Case.check for sigmoids that fp32 does not hold.  A score below 2^-126 is
    0 (of a row that is taken relative to its largest logit: below 2^-126 of that
    one's), so a share p is off by up to 2^-126 / sum of the scores beside its
    rounding; a gradient entry by that times |coef| (max count + sum p count), a
    weight's part by that, over the selected, times |g| + sum |g| w."""
    counts, tokens, P, loss = (t.cpu().numpy() for t in c.forward())
    wc, wt, wP, wl = loss64(c.l, c.ids, c.k, c.off, "sigmoid")
    np.testing.assert_array_equal(counts, wc)
    np.testing.assert_array_equal(tokens, wt)

    def flush(total):
        return 2.0 ** -126 / np.where(total < 2.0 ** -31, 1.0, total)
    sc, p = scores64(c.l, "sigmoid")
    lost = flush(sc.sum(axis=1, keepdims=True))
    rel = (c.E / 32 + 16 + 2 * np.abs(c.l).max() + chunk_bound(c.T) / 8 + 14) * U
    np.testing.assert_allclose(P, wP, rtol=rel, atol=c.T * lost.max())
    np.testing.assert_allclose(loss, wl, rtol=rel, atol=1e-37)
    seq = np.clip(np.searchsorted(c.off, np.arange(c.T), side="right") - 1, 0, c.S - 1)
    n = wc[seq].astype(np.float64)
    coef = np.abs(c.gl[seq]) * c.E / (c.k * np.maximum(wt[seq], 1).astype(np.float64) ** 2)
    slack = coef[:, None] * (n.max(axis=1, keepdims=True) + (p * n).sum(axis=1, keepdims=True)) * lost
    w, _, ok = weights64(c.l, c.ids, c.k, "sigmoid")
    sel = np.where(ok, np.take_along_axis(sc, np.clip(c.ids[:, :c.k], 0, c.E - 1), axis=1), 0).sum(axis=1, keepdims=True)
    g = np.abs(np.where(ok, c.gw, 0)).astype(np.float64)
    part = c.k * (g.max(axis=1, keepdims=True) + (g * w).sum(axis=1, keepdims=True)) * flush(sel)
    for gw in (True, False):
        got = c.backward(gw)
        want, err = grad64(c.l, c.ids, c.k, c.off, "sigmoid", c.gl, c.gw if gw else None)
        bad = np.abs(got - want) > err * U + slack + (part if gw else 0) + 1e-37
        assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], (err * U)[bad][:4])
    return counts, tokens, P, loss


@pytest.mark.parametrize("T,E,k", [(60, 72, 4), (33, 130, 6), (700, 384, 6), (300, 48, 6), (21, 1023, 7)])
def test_sigmoids_far_below_one(T, E, k):
    """Rows of which every sigmoid is below what fp32 holds, or close to it:
    their shares are well defined, those of e^l.  Logits around -88, -150 and
    around the border where rows are taken relative to their largest logit."""
    for lo, hi in ((-95, -80), (-160, -140), (-27, -18), (-120, 3)):
        c = Case(T, E, k, S=2, scoring="sigmoid", seed=E - hi, pad=0.1)
        c.l = np.random.default_rng(-lo).uniform(lo, hi, (T, E)).astype(np.float32)
        c.l[::5] += 100.0                                # ordinary rows between them
        counts, tokens, P, loss = check_low(c)
        assert (P[tokens > 0].sum(axis=1) > 0.999 * tokens[tokens > 0]).all()


@pytest.mark.parametrize("T,E,k", [(50, 64, 4), (700, 130, 6)])
def test_sigmoids_of_very_low_logits(T, E, k):
    """Around -2000 a sigmoid is e^l to any accuracy, so the sigmoid form is the
    softmax form; masked places among them stay without a share."""
    rng = np.random.default_rng(E)
    c = Case(T, E, k, S=2, scoring="sigmoid", seed=E)
    c.l = rng.normal(-2000, 2, (T, E)).astype(np.float32)
    m = rng.random((T, E)) < 0.3
    m[np.arange(T)[:, None], c.ids] = False
    for mask in (-np.inf, np.finfo(np.float32).min):
        c.l[m] = mask
        low = np.where(m, -np.inf, c.l).astype(np.float32)
        counts, tokens, P, loss = (t.cpu().numpy() for t in c.forward())
        wc, wt, wP, wl = loss64(low, c.ids, k, c.off, "softmax")
        np.testing.assert_array_equal(counts, wc)
        rel = (E / 32 + 16 + 60 + chunk_bound(T) / 8 + 14) * U       # logits of a row are within 30
        np.testing.assert_allclose(P, wP, rtol=rel, atol=1e-37)
        np.testing.assert_allclose(loss, wl, rtol=rel, atol=1e-37)
        for gw in (True, False):
            got = c.backward(gw)
            want, err = grad64(low, c.ids, k, c.off, "softmax", c.gl, c.gw if gw else None)
            assert (want != 0).any() and (np.abs(got - want) <= err * U + 1e-37).all()


def test_slots_far_below_the_rest_of_their_row():
    """The selected experts' sigmoids vanish beside the row's others: the
    weights among them are still those of their logits."""
    c = Case(80, 40, 4, S=2, scoring="sigmoid", seed=3)
    rng = np.random.default_rng(3)
    at = np.arange(80)[:, None]
    c.l[at, c.ids] = rng.uniform(-130, -90, (80, 4)).astype(np.float32)
    c.ids[::7, 1] = -1
    c.ids[::9, 2] = c.ids[::9, 0]
    check_low(c)


@pytest.mark.parametrize("E,k", [(8, 2), (130, 4), (384, 6), (1000, 8)])
def test_sums_of_sigmoids_at_the_border(E, k):
    """Rows whose sigmoids add up to 2^-30 within a few roundings, where one
    form of a row gives way to another: each row is counted once."""
    T = 600
    c = Case(T, E, k, S=2, scoring="sigmoid", seed=E)
    l = np.random.default_rng(E).normal(0, 1, (T, E))
    sums = np.exp(l).sum(axis=1, keepdims=True)
    c.l = (l - np.log(sums) - 30 * np.log(2.0) + np.linspace(-4e-6, 4e-6, T)[:, None]).astype(np.float32)
    counts, tokens, P, loss = check_low(c)
    assert np.abs(P.sum(axis=1) - tokens).max() < 1e-3 * T


def test_one_workspace_for_all_batch_lengths():
    """Sized for the longest batch, with no shorter one refused, and the same
    results as on a workspace of their own."""
    ws = torch.empty(nvfp4_moe_balance_workspace_size(3000, 4, 384), dtype=torch.uint8, device=DEV)
    for T, S in ((2048, 1), (2000, 0), (2049, 1), (3000, 4), (17, 2), (1500, 3)):
        c = Case(T, 384, 6, S=S, seed=T)
        l, ids, o = c.dev()
        out = [torch.empty(c.S, 384, dtype=torch.int32, device=DEV), torch.empty(c.S, dtype=torch.int32, device=DEV),
               torch.empty(c.S, 384, device=DEV), torch.empty(c.S, device=DEV)]
        nvfp4_moe_balance(l, ids, 6, *out, ws, seq_offsets=o)
        for a, b in zip(out, c.forward()):
            assert torch.equal(a, b)
