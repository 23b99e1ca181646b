"""The gradients through the packed head (logits_grad, nll_grad) against FP64 on the decoded
head, over formats, ranks, group sizes, odd sizes, masks, and as a whole training step with the
losses.

Tolerances, from the arithmetic.  A value is rounded to BF16 at the end (half a step: 2^-8
relative).  Before that each dY entry and each low-rank factor entry is rounded once to FP16
(2^-11 each) and sums are FP32: at most 2^-10 (1 + 2^-3) of sum_v |dY_v| |W|_vd, with |W| the
sum of the magnitudes of the residual and of the factors' products.  nll_grad's dY comes from
logits whose own error is bounded by 1e-4 max|Y| in the logits' tests, so that much
more of each probability.
FP16 also has a smallest step, 2^-24.  The product takes dY'[n, v] = dY[n, v] S'_v 2^e, S'_v the
row's scale (row_scale below) and 2^e such that the largest possible entry, max|dY[n]| max S',
lies between 2^12 and 2^14: half a step, 2^-25, is at most 2^-37 of that maximum, and it meets
the entry W_vd / S'_v.  So 2^-37 max|dY[n]| sum_v |W|_vd max S' / S'_v comes to the bound: it shows
only where everything larger in the row meets weights of exactly 0."""
import ctypes
import os

import numpy as np
import pytest
import torch

import oracle
import packed_int4_lm_b200 as ah
from packed_int4_lm_b200 import _lib
from packed_int4_lm_b200._lib import STATUS_CODE as E
from workloads import bf16_bits, make_channel_scales, make_hidden, make_targets, random_canonical_head

BF16, PROD = 2.0 ** -8, 2.0 ** -10 * 1.125


def row8_head(V, D, seed):
    rng = np.random.default_rng(seed)
    return {"format": "row8", "V": V, "D": D, "r_c": 0, "r_r": 0, "g": 128,
            "q8": rng.integers(-127, 128, size=(V, D)).astype(np.int8),
            "row_scale": (2.0 ** rng.uniform(-13, -11, size=V)).astype(np.float32)}


def make_head(V, D, r_c, r_r, g, seed=1, **kw):
    """Random bytes with logits of a few units."""
    kw = {"super_exp_range": (-17, -13), "factor_exp_range": (-13, -10), "zero_rows": 2, **kw}
    return random_canonical_head(V, D, r_c, r_r, g, seed=seed, **kw)


def magnitudes(head):
    """W and sum of the magnitudes that make it up, FP64."""
    W = oracle.dense_head_rows(head)
    if head.get("format") == "row8":
        return W, np.abs(W)
    M = np.abs(oracle.unpack_residual(head))
    for a, b in (("Ac", "Bc"), ("Aw", "Bw")):
        if head[a].shape[1]:
            M = M + np.abs(oracle.dequant_int8_rowwise(head[a], head["s" + a])) @ np.abs(
                oracle.dequant_int8_groupwise(head[b], head["s" + b], head["g"]))
    return W, M


def row_scale(head):
    """S'_v: the scale in units of which a row of the head is held in FP16."""
    if head.get("format") == "row8":
        return head["row_scale"].astype(np.float64)
    S = oracle.bf16_bits_to_f64(head["r_super"])
    m = 128 * np.maximum(head["sAc"] * (head["r_c"] > 0), head["sAw"] * (head["r_r"] > 0)).astype(np.float64)
    log = lambda x: np.floor(np.log2(np.where(x > 0, x, 1)))
    k = np.maximum(log(m) - log(S) - 13, -3)
    return np.where(m == 0, S, np.where((S == 0) | (k > 40), 2.0 ** (log(m) - 13), S * 2.0 ** k))


def smallest_step(head, M, dY):
    """The bound's last term, N x D."""
    s = row_scale(head)
    share = np.divide(s.max(), s, out=np.zeros_like(s), where=s > 0)
    return 2.0 ** -37 * np.abs(dY.astype(np.float64)).max(1, keepdims=True) * (share @ M)


def close(got, want, tol, what=""):
    got = got.cpu().double().numpy()
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3],
                           want[bad][:3], tol[bad][:3])


HEADS = {
    "g64": lambda: make_head(1000, 512, 8, 8, 64),
    "g32 odd": lambda: make_head(1237, 640, 7, 18, 32),
    "g128": lambda: make_head(4099, 384, 32, 32, 128),
    "g256 ranks 128": lambda: make_head(777, 768, 128, 128, 256),
    "no ranks": lambda: make_head(513, 128, 0, 0, 128),
    "core only": lambda: make_head(260, 256, 20, 0, 64),
    "one row": lambda: make_head(1, 128, 3, 0, 32, zero_rows=0),
    "wide scales": lambda: make_head(900, 256, 16, 16, 128, super_exp_range=(-22, -8),
                                     factor_exp_range=(-14, -9)),
    "row8": lambda: row8_head(1000, 512, 3),
    "row8 odd": lambda: row8_head(333, 640, 4),
}
_cache = {}


def head_of(name):
    if name not in _cache:
        h = HEADS[name]()
        _cache[name] = (h, *magnitudes(h))
    return _cache[name]


def make_dY(N, V, seed):
    """A softmax gradient's shape: small positives and one large negative, rows of very
    different size, one row of zeros."""
    rng = np.random.default_rng(seed)
    y = np.exp(2.5 * rng.normal(size=(N, V)))
    y /= y.sum(1, keepdims=True)
    y[np.arange(N), rng.integers(0, V, size=N)] -= 1
    y *= 2.0 ** rng.integers(-30, 20, size=(N, 1))
    if N > 2:
        y[1] = 0
    return y.astype(np.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("name", HEADS, ids=str)
@pytest.mark.parametrize("N", [1, 7, 16, 17, 33, 100, 130, 300, 600])
def test_logits_grad_matches_fp64(cuda_ok, name, N):
    head, W, M = head_of(name)
    dh = ah.DeviceHead.from_canonical(head, "cuda")
    dY = make_dY(N, head["V"], 10 + N)
    got = ah.logits_grad(torch.from_numpy(dY).cuda(), dh)
    ah.check()
    want = dY.astype(np.float64) @ W
    close(got, want, BF16 * np.abs(want) + PROD * (np.abs(dY).astype(np.float64) @ M)
          + smallest_step(head, M, dY), name)


@pytest.mark.gpu
@pytest.mark.parametrize("D,r,g", [(4096, 32, 128), (3968, 40, 32)])
def test_few_tokens_through_a_large_head(cuda_ok, D, r, g):
    """Slabs of the vocabulary longer than a kernel's ring of stages, in up to 8 and more tokens;
    every row has the same bits whatever the batch beside it."""
    head = make_head(23017, D, r, r, g)
    W, M = magnitudes(head)
    dh = ah.DeviceHead.from_canonical(head, "cuda")
    dY = make_dY(9, head["V"], D)
    want = dY.astype(np.float64) @ W
    tol = BF16 * np.abs(want) + PROD * (np.abs(dY).astype(np.float64) @ M) + smallest_step(head, M, dY)
    t = torch.from_numpy(dY).cuda()
    rows = {}
    for N in (9, 8, 5, 1):
        got = rows[N] = ah.logits_grad(t[:N], dh)
        ah.check()
        close(got, want[:N], tol[:N], N)
    assert torch.equal(rows[8][:5], rows[5]) and torch.equal(rows[5][:1], rows[1])


def nll_case(head, W, N, seed):
    D, V = head["D"], head["V"]
    H = make_hidden(N, make_channel_scales(D, 0.5, 4, 20.0, seed), seed + 1)
    tg = make_targets(N, V, seed + 2).numpy()
    Y = oracle.logits(head, bf16_bits(H))
    m = Y.max(1)
    lse = m + np.log(np.exp(Y - m[:, None]).sum(1))
    P = np.exp(Y - lse[:, None])
    P[np.arange(N), tg] = np.expm1(Y[np.arange(N), tg] - lse)
    dnll = np.random.default_rng(seed + 3).normal(size=N) * 2.0 ** (seed % 7 - 3)
    return H, tg, Y, lse, P, dnll.astype(np.float32)


def nll_tol(head, P, Y, M, dnll, want):
    d = np.abs(dnll.astype(np.float64))[:, None]
    return (BF16 * np.abs(want) + (PROD + 1e-4 * np.abs(Y).max()) * d * (np.abs(P) @ M)
            + d * smallest_step(head, M, P))


@pytest.mark.gpu
@pytest.mark.parametrize("name", [h for h in HEADS if h != "one row"], ids=str)
@pytest.mark.parametrize("N", [1, 16, 17, 64, 130, 300])
def test_nll_grad_matches_fp64(cuda_ok, name, N):
    head, W, M = head_of(name)
    dh = ah.DeviceHead.from_canonical(head, "cuda")
    H, tg, Y, lse, P, dnll = nll_case(head, W, N, 30 + N)
    masked = np.arange(N) % 5 == 3
    dnll[masked] = 0
    Hd, t = H.cuda(), torch.from_numpy(tg).cuda()
    nl, ls = ah.nll_lse(Hd, dh, t)
    assert torch.equal(nl, ah.nll(Hd, dh, t))
    # no logit is off by more than 1e-4 max|Y| (the logits' own tests), and a log-sum-exp moves
    # by at most the largest change of a logit
    assert np.abs(ls.cpu().double().numpy() - lse).max() <= 1e-4 * np.abs(Y).max()
    t[torch.from_numpy(masked).cuda()] = -100  # masked tokens need no target
    nl[torch.from_numpy(masked).cuda()] = float("nan")
    dev = torch.from_numpy(dnll).cuda()
    got = ah.nll_grad(Hd, dh, t, nl, ls, dev)
    ah.check()
    want = dnll.astype(np.float64)[:, None] * (P @ W)
    close(got, want, nll_tol(head, P, Y, M, dnll, want), name)
    assert not got[torch.from_numpy(masked).cuda()].any()
    assert torch.equal(got, ah.nll_grad(Hd, dh, t, nl, ls, dev))  # equal calls, equal bits


@pytest.mark.gpu
@pytest.mark.parametrize("name,N", [("g128", 2331), ("g64", 9500), ("g32 odd", 7700), ("g256 ranks 128", 9729),
                                    ("core only", 38000), ("wide scales", 9600)])
def test_nll_grad_of_large_batches(cuda_ok, name, N):
    """Batches that run in tiles of 256 tokens x 256 rows, the last ones ragged: 240 of their
    tokens, the last tile's among them, against FP64."""
    head, W, M = head_of(name)
    dh = ah.DeviceHead.from_canonical(head, "cuda")
    V, D = head["V"], head["D"]
    rng = np.random.default_rng(N)
    rows = np.unique(np.r_[rng.integers(0, N, size=160), N - 80:N])
    H = make_hidden(N, make_channel_scales(D, 0.5, 4, 20.0, 1), 2)
    tg = make_targets(N, V, 3).numpy()
    dnll = rng.normal(size=N).astype(np.float32)
    dnll[rows[::7]] = 0
    t = torch.from_numpy(tg).cuda()
    Hd = H.cuda()
    nl, ls = ah.nll_lse(Hd, dh, t)
    dn = torch.from_numpy(dnll).cuda()
    got = ah.nll_grad(Hd, dh, t, nl, ls, dn)
    ah.check()
    assert torch.equal(got, ah.nll_grad(Hd, dh, t, nl, ls, dn))
    Y = oracle.logits(head, bf16_bits(H[rows]))
    m = Y.max(1)
    lse = m + np.log(np.exp(Y - m[:, None]).sum(1))
    P = np.exp(Y - lse[:, None])
    at = (np.arange(len(rows)), tg[rows])
    P[at] = np.expm1(Y[at] - lse)
    want = dnll[rows].astype(np.float64)[:, None] * (P @ W)
    close(got[torch.from_numpy(rows).cuda()], want, nll_tol(head, P, Y, M, dnll[rows], want), name)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [9, 40, 200])
def test_nll_grad_of_confident_tokens(cuda_ok, N):
    """Targets whose probability is close to 1: the gradient is a small difference, which must
    keep its relative precision per token."""
    head, W, M = head_of("g64")
    dh = ah.DeviceHead.from_canonical(head, "cuda")
    D = head["D"]
    rng = np.random.default_rng(3)
    tg = rng.integers(0, head["V"], size=N).astype(np.int32)
    # hidden states along the target's row: its logit leads by 2 to 16
    base = W[tg] / (W[tg] ** 2).sum(1, keepdims=True) * np.linspace(8, 30, N)[:, None]
    H = torch.from_numpy(base + 0.3 * rng.normal(size=(N, D))).to(torch.bfloat16)
    Y = oracle.logits(head, bf16_bits(H))
    m = Y.max(1)
    lse = m + np.log(np.exp(Y - m[:, None]).sum(1))
    P = np.exp(Y - lse[:, None])
    rest = P.copy()
    rest[np.arange(N), tg] = 0
    P[np.arange(N), tg] = -rest.sum(1)
    Hd, t = H.cuda(), torch.from_numpy(tg).cuda()
    nl, ls = ah.nll_lse(Hd, dh, t)
    got = ah.nll_grad(Hd, dh, t, nl, ls, torch.ones(N, device="cuda"))
    ah.check()
    want = P @ W
    # the NLL and the log-sum-exp are FP32 values: each is off by up to 4 half steps of the
    # largest logit, so every probability by that much relative, and the target's entry
    # 1 - p by as much of p
    slip = 4 * 2.0 ** -24 * np.abs(Y).max(1)[:, None]
    tol = nll_tol(head, P, Y, M, np.ones(N, np.float32), want) + 2 * slip * M[tg]
    close(got, want, tol)
    assert nl.min() < 1e-3  # such tokens were there


@pytest.mark.gpu
def test_nll_grad_against_differences(cuda_ok):
    """The directional derivative of sum dnll * NLL by differences of the FP64 oracle."""
    head, W, M = head_of("g128")
    dh = ah.DeviceHead.from_canonical(head, "cuda")
    N = 48
    H, tg, Y, lse, P, dnll = nll_case(head, W, N, 77)
    Hd, t = H.cuda(), torch.from_numpy(tg).cuda()
    nl, ls = ah.nll_lse(Hd, dh, t)
    got = ah.nll_grad(Hd, dh, t, nl, ls, torch.from_numpy(dnll).cuda()).cpu().double().numpy()
    ah.check()
    H64 = H.double().numpy()
    want = dnll.astype(np.float64)[:, None] * (P @ W)
    tol = nll_tol(head, P, Y, M, dnll, want)
    for seed in range(4):
        u = np.random.default_rng(seed).normal(size=H64.shape)
        f = [(dnll * oracle.nll_from_logits((H64 + s * u) @ W.T, tg)).sum() for s in (1e-5, -1e-5)]
        assert abs((f[0] - f[1]) / 2e-5 - (got * u).sum()) <= (tol * np.abs(u)).sum() * 0.2 + 1e-6


@pytest.mark.gpu
def test_bad_targets_and_non_finite_rows_stay_in_their_rows(cuda_ok):
    head, W, M = head_of("g64")
    dh = ah.DeviceHead.from_canonical(head, "cuda")
    for N in (5, 70, 280):
        H, tg, Y, lse, P, dnll = nll_case(head, W, N, 5)
        dnll[dnll == 0] = 1
        Hd, t = H.cuda(), torch.from_numpy(tg).cuda()
        nl, ls = ah.nll_lse(Hd, dh, t)
        dn = torch.from_numpy(dnll).cuda()
        good = ah.nll_grad(Hd, dh, t, nl, ls, dn)
        t[2], t[4] = head["V"], -1
        got = ah.nll_grad(Hd, dh, t, nl, ls, dn)
        with pytest.raises(ah.ArcheadError) as e:
            ah.check()
        assert e.value.status == E["ARCHEAD_ERR_TARGET"]
        assert torch.isnan(got[[2, 4]]).all()
        keep = [n for n in range(N) if n not in (2, 4)]
        assert torch.equal(got[keep], good[keep])
        dY = torch.from_numpy(make_dY(N, head["V"], 9)).cuda()
        good = ah.logits_grad(dY, dh)
        dY[2, 17], dY[4, 999] = float("nan"), float("inf")
        got = ah.logits_grad(dY, dh)
        ah.check()
        assert not torch.isfinite(got[[2, 4]]).any()
        assert torch.equal(got[keep], good[keep])


@pytest.mark.gpu
@pytest.mark.parametrize("N", [3, 70, 300])
def test_outputs_stay_inside_their_rows(cuda_ok, N):
    """Guard bands around dH are untouched, on a vocabulary and batch that end inside tiles."""
    head, W, M = head_of("g32 odd")
    dh = ah.DeviceHead.from_canonical(head, "cuda")
    D = head["D"]
    H, tg, Y, lse, P, dnll = nll_case(head, W, N, 6)
    Hd, t = H.cuda(), torch.from_numpy(tg).cuda()
    nl, ls = ah.nll_lse(Hd, dh, t)
    dY = torch.from_numpy(make_dY(N, head["V"], 9)).cuda()
    for call in (lambda o: ah.nll_grad(Hd, dh, t, nl, ls, torch.from_numpy(dnll).cuda(), out=o),
                 lambda o: ah.logits_grad(dY, dh, out=o)):
        buf = torch.full((N + 64, D), float("nan"), device="cuda", dtype=torch.bfloat16)
        call(buf[32:32 + N])
        ah.check()
        assert torch.isnan(buf[:32]).all() and torch.isnan(buf[32 + N:]).all()
        assert torch.isfinite(buf[32:32 + N]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("N", [12, 150])
def test_training_step_of_the_operators_together(cuda_ok, N):
    """Forward, policy loss or preference loss, and the way back to the hidden states, as a user
    chains them, on another stream than the current one and captured into a graph, against FP64
    autograd through the dense head."""
    head, W, M = head_of("g64")
    dh = ah.DeviceHead.from_canonical(head, "cuda")
    H, tg, Y, lse, P, _ = nll_case(head, W, N, 40)
    rng = np.random.default_rng(1)
    cu = np.array([0, N // 3, N // 3, N // 2, N], dtype=np.int32)
    pairs = np.array([[0, 3], [2, 3], [0, 2]], dtype=np.int32)
    w = (np.arange(N) % 4 != 1).astype(np.float32)
    true = lse - Y[np.arange(N), tg]
    old = (true + 0.05 * rng.normal(size=N)).astype(np.float32)
    ref = (true + 0.2 * rng.normal(size=N)).astype(np.float32)
    adv = rng.normal(size=4).astype(np.float32)
    dev = {k: torch.from_numpy(v).cuda() for k, v in
           dict(tg=tg, cu=cu, pairs=pairs, w=w, old=old, ref=ref, adv=adv).items()}
    Hd = H.cuda()

    def step(which, stream=None):
        nl, ls = ah.nll_lse(Hd, dh, dev["tg"], stream=stream)
        if which == "policy":
            out = ah.policy_loss(nl, dev["old"], dev["adv"], nll_ref=dev["ref"], weights=dev["w"],
                                 cu_seqlens=dev["cu"], per_sequence=True, kl_coef=0.2,
                                 reduction="sequence", clip_low=0.9, clip_high=9.0, stream=stream)
        else:
            out = ah.preference_loss(nl, dev["cu"], dev["pairs"], nll_ref=dev["ref"],
                                     weights=dev["w"], beta=0.3, stream=stream)
        return ah.nll_grad(Hd, dh, dev["tg"], nl, ls, out["dnll"], stream=stream), out["dnll"]

    for which in ("policy", "preference"):
        got, dnll = step(which)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        other, _ = step(which, stream=side)
        side.synchronize()
        assert torch.equal(got, other)
        g = torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=side):
            cap, _ = step(which)
        g.replay()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, cap)
        ah.check()
        # the same step in FP64 through autograd
        x = H.double().requires_grad_()
        y = x @ torch.from_numpy(W).T
        nl = torch.logsumexp(y, 1) - y[torch.arange(N), torch.from_numpy(tg).long()]
        W64 = torch.from_numpy(w).double()
        seg = [slice(cu[i], cu[i + 1]) for i in range(4)]
        if which == "policy":
            r, z = torch.exp(torch.from_numpy(old) - nl), nl - torch.from_numpy(ref)
            a = torch.from_numpy(adv).double()[torch.repeat_interleave(torch.arange(4), torch.from_numpy(np.diff(cu)))]
            l = -torch.minimum(r * a, r.clamp(0.1, 10) * a) + 0.2 * (torch.expm1(z) - z)
            loss = sum((W64 * l)[s].sum() / W64[s].sum() for s in (seg[0], seg[2], seg[3])) / 3
        else:
            f = torch.stack([(W64 * (torch.from_numpy(ref) - nl))[s].sum() for s in seg])
            loss = -torch.nn.functional.logsigmoid(0.3 * (f[pairs[:, 0]] - f[pairs[:, 1]])).mean()
        loss.backward()
        want = x.grad.numpy()
        d = dnll.cpu().numpy()
        # dnll comes from FP32 NLLs off by up to 1e-4 max|Y| each (as logits are), which moves a
        # ratio, and a pair's score by the sum over its tokens, by that much relative
        slip = 1e-4 * np.abs(Y).max() * (2 if which == "policy" else 1 + 0.3 * N) * np.abs(d).max()
        close(got, want, nll_tol(head, P, Y, M, d, want) + slip * (np.abs(P) @ M), which)


@pytest.mark.gpu
@pytest.mark.parametrize("extra", [5, 40])
def test_batches_beyond_one_chunk(cuda_ok, extra):
    """More tokens than one pass takes (65536), with a last pass of another size, which may run on
    another kernel: rows of the first, the middle and the last tokens against FP64."""
    head, W, M = head_of("no ranks")
    dh = ah.DeviceHead.from_canonical(head, "cuda")
    V, D = head["V"], head["D"]
    N = 2 * 65536 + extra
    rows = np.r_[0:6, 65530:65542, N - extra - 3:N]
    H = make_hidden(N, make_channel_scales(D, 0.5, 4, 20.0, 1), 2)
    t = make_targets(N, V, 3).cuda()
    Hd = H.cuda()
    nl, ls = ah.nll_lse(Hd, dh, t)
    dn = torch.linspace(-1, 1, N, device="cuda")
    got = ah.nll_grad(Hd, dh, t, nl, ls, dn)[torch.from_numpy(rows).cuda()]
    ah.check()
    Y = oracle.logits(head, bf16_bits(H[rows]))
    m = Y.max(1)
    lse = m + np.log(np.exp(Y - m[:, None]).sum(1))
    P = np.exp(Y - lse[:, None])
    at = t.cpu().numpy()[rows]
    P[np.arange(len(rows)), at] = np.expm1(Y[np.arange(len(rows)), at] - lse)
    d = dn.cpu().numpy()[rows]
    want = d.astype(np.float64)[:, None] * (P @ W)
    close(got, want, nll_tol(head, P, Y, M, d, want), "nll_grad")
    dY = torch.randn(N, V, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    got = ah.logits_grad(dY, dh)[torch.from_numpy(rows).cuda()]
    ah.check()
    y = dY[torch.from_numpy(rows).cuda()].cpu().numpy()
    want = y.astype(np.float64) @ W
    close(got, want, BF16 * np.abs(want) + PROD * (np.abs(y).astype(np.float64) @ M) + smallest_step(head, M, y))


@pytest.mark.gpu
@pytest.mark.parametrize("N", [3, 140])
def test_dY_aligned_to_four_bytes_only(cuda_ok, N):
    head, W, M = head_of("g64")
    dh = ah.DeviceHead.from_canonical(head, "cuda")
    dY = torch.from_numpy(make_dY(N, head["V"], 8)).cuda()
    buf = torch.empty(N * head["V"] + 1, device="cuda")
    off = buf[1:].view(N, head["V"])
    off.copy_(dY)
    assert off.data_ptr() % 16 == 4
    assert torch.equal(ah.logits_grad(off, dh), ah.logits_grad(dY, dh))
    ah.check()


@pytest.mark.gpu
@pytest.mark.parametrize("N", [5, 60, 300])
def test_negative_super_scales_and_rows_of_zeros(cuda_ok, N):
    """The format allows a negative super-scale; rows of nothing (no residual, zero factors)."""
    head = make_head(700, 256, 16, 16, 64, seed=5)
    head["r_super"][::3] |= 0x8000
    head["r_super"][7:40] = 0
    head["sAc"][20:30] = 0
    head["sAw"][20:40] = 0
    W, M = magnitudes(head)
    dh = ah.DeviceHead.from_canonical(head, "cuda")
    dY = make_dY(N, 700, 4)
    got = ah.logits_grad(torch.from_numpy(dY).cuda(), dh)
    want = dY.astype(np.float64) @ W
    pos = {**head, "r_super": head["r_super"] & np.uint16(0x7FFF)}
    close(got, want, BF16 * np.abs(want) + PROD * (np.abs(dY).astype(np.float64) @ M) + smallest_step(pos, M, dY))
    H, tg, Y, lse, P, dnll = nll_case(head, W, N, 9)
    Hd, t = H.cuda(), torch.from_numpy(tg).cuda()
    nl, ls = ah.nll_lse(Hd, dh, t)
    got = ah.nll_grad(Hd, dh, t, nl, ls, torch.from_numpy(dnll).cuda())
    ah.check()
    want = dnll.astype(np.float64)[:, None] * (P @ W)
    close(got, want, nll_tol(pos, P, Y, M, dnll, want))


@pytest.mark.gpu
def test_two_streams_at_once(cuda_ok):
    """Calls in flight on two streams do not share scratch."""
    head, W, M = head_of("g128")
    dh = ah.DeviceHead.from_canonical(head, "cuda")
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    dY = [torch.from_numpy(make_dY(200, head["V"], k)).cuda() for k in range(2)]
    want = [ah.logits_grad(y, dh) for y in dY]
    torch.cuda.synchronize()
    got = [ah.logits_grad(dY[i % 2], dh, stream=s[i % 2]) for i in range(12)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 2]) for i, g in enumerate(got))
    ah.check()


@pytest.mark.gpu
def test_no_tokens(cuda_ok):
    head, W, M = head_of("g64")
    dh = ah.DeviceHead.from_canonical(head, "cuda")
    e = torch.empty(0, device="cuda")
    H = torch.empty(0, head["D"], device="cuda", dtype=torch.bfloat16)
    t = e.to(torch.int32)
    assert ah.nll_grad(H, dh, t, e, e, e).shape == (0, head["D"])
    assert ah.logits_grad(torch.empty(0, head["V"], device="cuda"), dh).shape == (0, head["D"])
    assert [x.shape for x in ah.nll_lse(H, dh, t)] == [(0,), (0,)]
    ah.check()


@pytest.mark.gpu
def test_binding_checks(cuda_ok):
    head, W, M = head_of("g64")
    dh = ah.DeviceHead.from_canonical(head, "cuda")
    V, D = head["V"], head["D"]
    dY = torch.zeros(4, V, device="cuda")
    for bad in (dY.cpu(), dY.double(), dY[:, :-1], torch.zeros(V, 4, device="cuda").t(), dY[0]):
        with pytest.raises(ValueError):
            ah.logits_grad(bad, dh)
    for out in (torch.empty(4, D, device="cuda"), torch.empty(3, D, device="cuda", dtype=torch.bfloat16),
                torch.empty(D, 4, device="cuda", dtype=torch.bfloat16).t()):
        with pytest.raises(ValueError):
            ah.logits_grad(dY, dh, out=out)
    H = torch.zeros(4, D, device="cuda", dtype=torch.bfloat16)
    t = torch.zeros(4, device="cuda", dtype=torch.int32)
    f = torch.zeros(4, device="cuda")
    good = dict(targets=t, nll=f, lse=f, dnll=f)
    for k, bad in (("targets", t.long()), ("targets", t[:3]), ("nll", f.double()), ("lse", f[:3]),
                   ("dnll", f.cpu()), ("dnll", torch.zeros(8, device="cuda")[::2])):
        with pytest.raises(ValueError):
            ah.nll_grad(H, dh, **{**good, k: bad})
    with pytest.raises(ValueError):
        ah.nll_grad(H.float(), dh, **good)
    with pytest.raises(ValueError):
        ah.nll_lse(H, dh, t[:3])


# ---- refusals (host) --------------------------------------------------------------------
def test_gradient_argument_errors():
    if not os.path.exists(_lib.LIB_PATH):
        from packed_int4_lm_b200 import build
        build.build()
    L = _lib.lib()
    h = _lib.ArcheadHead()
    h.V, h.D, h.r_c, h.r_r, h.g = 1000, 512, 4, 4, 64
    for i, k in enumerate(("r_nib", "r_code", "r_super", "Ac", "sAc", "Bc", "sBc", "Aw", "sAw",
                           "Bw", "sBw")):
        setattr(h, k, 0x100000 * (i + 1))
    a = 0x9000000

    def nll_grad(H=a, head=h, t=a, nll=a, lse=a, dn=a, dH=a, N=4, V=1000):
        return L.archead_nll_grad(H, ctypes.byref(head) if head else None, t, nll, lse, dn, dH, N, V,
                                  512, 4, 4, 64, None)

    def logits_grad(dY=a, head=h, dH=a, N=4, D=512):
        return L.archead_logits_grad(dY, ctypes.byref(head) if head else None, dH, N, 1000, D, 4, 4,
                                     64, None)

    def nll_lse(nll=a, lse=a, N=4):
        return L.archead_nll_lse(a, ctypes.byref(h), a, nll, lse, N, 1000, 512, 4, 4, 64, None)

    for got, code in (
            (nll_grad(H=None), "NULLPTR"), (nll_grad(head=None), "NULLPTR"),
            (nll_grad(t=None), "NULLPTR"), (nll_grad(nll=None), "NULLPTR"),
            (nll_grad(lse=None), "NULLPTR"), (nll_grad(dn=None), "NULLPTR"),
            (nll_grad(dH=None), "NULLPTR"), (nll_grad(H=a + 8), "ALIGN"),
            (nll_grad(dH=a + 8), "ALIGN"), (nll_grad(dn=a + 2), "ALIGN"),
            (nll_grad(N=-1), "SHAPE"), (nll_grad(V=999), "SHAPE"),
            (logits_grad(dY=None), "NULLPTR"), (logits_grad(dH=None), "NULLPTR"),
            (logits_grad(head=None), "NULLPTR"), (logits_grad(dY=a + 1), "ALIGN"),
            (logits_grad(dH=a + 4), "ALIGN"), (logits_grad(D=500), "SHAPE"),
            (logits_grad(N=1 << 31), "SHAPE"),
            (nll_lse(nll=None), "NULLPTR"), (nll_lse(lse=None), "NULLPTR"),
            (nll_lse(lse=a + 2), "ALIGN"), (nll_lse(N=-2), "SHAPE")):
        assert got == E["ARCHEAD_ERR_" + code], code
    assert nll_grad(N=0) == logits_grad(N=0) == nll_lse(N=0) == E["ARCHEAD_OK"]
