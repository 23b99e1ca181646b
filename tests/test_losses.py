"""The losses on per-token NLLs (policy_loss, preference_loss): value and gradient against
plain FP64 NumPy formulas, their gradients against differences of those formulas, masks,
empty and ragged sequences, refusals, streams and graphs."""
import ctypes
import os

import numpy as np
import pytest
import torch

import packed_int4_lm_b200 as ah
from packed_int4_lm_b200 import _lib
from packed_int4_lm_b200._lib import STATUS_CODE as E

U = 2.0 ** -24  # half a step of FP32, relative


# ---- FP64 formulas ----------------------------------------------------------------------
def seq_ids(cu, N):
    ids = np.full(N, -1)
    for i in range(len(cu) - 1):
        ids[cu[i]:cu[i + 1]] = i
    return ids


def policy_ref(nll, old, adv, ref=None, w=None, cu=None, per_seq=False, lo=0.2, hi=0.2, beta=0.0,
               reduction="token"):
    N = len(nll)
    ids = seq_ids(cu, N) if cu is not None else np.zeros(N, dtype=int)
    w = np.ones(N) if w is None else w.astype(np.float64)
    w = np.where(ids >= 0, w, 0.0)
    A = adv[np.maximum(ids, 0)] if per_seq else adv
    scale = np.zeros(N)
    if reduction == "sum":
        scale[:] = 1
    elif reduction == "token":
        scale[:] = 1 / w.sum() if w.sum() > 0 else 0
    else:
        tot = np.array([w[ids == i].sum() for i in range(len(cu) - 1)])
        for i in np.nonzero(tot > 0)[0]:
            scale[ids == i] = 1 / tot[i] / (tot > 0).sum()
    on = w != 0
    loss = sur = kl = clip = mag = 0.0
    grad, size = np.zeros(N), np.zeros(N)
    for n in np.nonzero(on)[0]:
        r = np.exp(float(old[n]) - float(nll[n]))
        a = float(A[n])
        kept = min(max(r, 1 - lo), 1 + hi)
        c = r * a > kept * a
        s = -min(r * a, kept * a)
        g = 0.0 if c else r * a
        z = float(nll[n]) - float(ref[n]) if ref is not None else 0.0
        k = np.expm1(z) - z
        f = w[n] * scale[n]
        sur, kl, clip = sur + f * s, kl + f * k, clip + f * c
        grad[n] = f * (g + beta * np.expm1(z))
        # |x| half steps of the difference inside exp, a few of exp and the products
        size[n] = f * ((abs(old[n] - nll[n]) + 8) * r * abs(a) * (not c) + beta * (abs(z) + 8) * (np.exp(z) + 1))
        mag += size[n] + f * abs(s) + f * k
    return {"stats": np.array([sur + beta * kl, sur, kl, clip]), "dnll": grad, "size": size, "mag": mag}


def preference_ref(nll, cu, pairs, ref=None, w=None, beta=0.1, kind="sigmoid", smooth=0.0, margin=0.0,
                   average=False):
    N, B = len(nll), len(cu) - 1
    w = np.ones(N) if w is None else w.astype(np.float64)
    x = np.where(w != 0, (0.0 if ref is None else ref.astype(np.float64)) - nll.astype(np.float64), 0.0)
    tot = np.array([w[cu[i]:cu[i + 1]].sum() for i in range(B)])
    f = np.array([(w * x)[cu[i]:cu[i + 1]].sum() for i in range(B)])
    per = np.divide(1.0, tot, out=np.zeros(B), where=tot > 0) if average else np.ones(B)
    f = f * per
    loss, back, size = [], np.zeros(B), np.zeros(B)
    for a, b in pairs:
        gap = f[a] - f[b]
        m = beta * gap - margin
        if kind == "sigmoid":
            l = (1 - smooth) * np.logaddexp(0, -m) + smooth * np.logaddexp(0, m)
            s = beta * (smooth / (1 + np.exp(-m)) - (1 - smooth) / (1 + np.exp(m)))
        elif kind == "hinge":
            l, s = max(0.0, 1 - m), -beta if m < 1 else 0.0
        else:
            d = gap - margin - 0.5 / beta
            l, s = d * d, 2 * d
        loss.append(l)
        back[a] += s / len(pairs)
        back[b] -= s / len(pairs)
        size[[a, b]] += abs(s) / len(pairs)
    grad = np.zeros(N)
    gsize = np.zeros(N)
    for i in range(B):
        grad[cu[i]:cu[i + 1]] = -w[cu[i]:cu[i + 1]] * back[i] * per[i]
        gsize[cu[i]:cu[i + 1]] = w[cu[i]:cu[i + 1]] * size[i] * per[i]
    p = np.array(pairs).reshape(-1, 2)
    return {"loss": np.array([np.mean(loss) if loss else 0.0]), "pair_loss": np.array(loss),
            "rewards": beta * np.stack([f[p[:, 0]], f[p[:, 1]]], 1), "dnll": grad, "size": gsize,
            "f": np.abs(w * x).sum()}


# ---- inputs -----------------------------------------------------------------------------
def offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


LENS = {
    "one token": [1],
    "one sequence": [300],
    "empty ones": [0, 0, 5, 0, 1, 0, 700, 0],
    "piece edges": [256, 255, 257, 1, 1024, 0, 512],
    "many short": [3, 0, 1, 2] * 300,
    "short in one block": [1] * 100 + [1, 2, 0, 3, 33, 1] * 20 + [0] * 70 + [2] * 100,
    "one long": [2, 20011, 1],
    "many": list(np.random.default_rng(5).integers(0, 40, size=1500)),
}


def make_tokens(N, seed, spread=0.3):
    rng = np.random.default_rng(seed)
    nll = np.abs(rng.normal(size=N) * 2).astype(np.float32)
    old = np.maximum(nll + spread * rng.normal(size=N), 0).astype(np.float32)
    ref = np.maximum(nll + spread * rng.normal(size=N), 0).astype(np.float32)
    w = rng.choice([0.0, 1.0, 1.0, 0.5], size=N).astype(np.float32)
    return nll, old, ref, w, rng


def cu_dev(*arrays):
    return [None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays]


def close(got, want, tol, what):
    got = got.cpu().double().numpy()
    assert got.shape == want.shape, what
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, got[bad][:3], want[bad][:3], np.broadcast_to(tol, want.shape)[bad][:3])


# ---- policy loss ------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("reduction", ["token", "sequence", "sum"])
@pytest.mark.parametrize("form", ["all", "plain", "per_seq"])
def test_policy_loss_matches_formula(cuda_ok, lens, reduction, form):
    cu = offsets(LENS[lens])
    N = int(cu[-1])
    nll, old, ref, w, rng = make_tokens(N, 11)
    per_seq = form == "per_seq"
    adv = rng.normal(size=len(cu) - 1 if per_seq else N).astype(np.float32)
    if form == "plain":
        ref = w = None
        if reduction != "sequence":
            cu = None
    if w is not None and len(LENS[lens]) > 3:
        w[cu[2]:cu[3]] = 0  # a sequence of which nothing counts
    kw = dict(lo=0.2, hi=0.3, beta=0.1)
    want = policy_ref(nll, old, adv, ref, w, cu, per_seq, reduction=reduction, **kw)
    if w is not None:  # masked places may hold anything
        for a in (nll, old, ref):
            a[w == 0] = rng.choice([np.nan, np.inf, -np.inf], size=int((w == 0).sum()))
    d = cu_dev(nll, old, adv, ref, w, cu)
    got = ah.policy_loss(d[0], d[1], d[2], nll_ref=d[3], weights=d[4], cu_seqlens=d[5],
                         per_sequence=per_seq, clip_low=0.2, clip_high=0.3, kl_coef=0.1,
                         reduction=reduction)
    ah.check()
    close(got["dnll"], want["dnll"], U * (want["size"] + np.abs(want["dnll"])), "dnll")
    close(got["stats"], want["stats"], 2 * U * (want["mag"] + np.abs(want["stats"])), "stats")


@pytest.mark.gpu
def test_policy_clip_border_and_infinite_ratios(cuda_ok):
    """Just inside, on and just outside the border; ratios that overflow; advantage zero."""
    old = np.float32(3.0)
    x = np.log1p(0.25)
    near = np.float32(old - x)
    steps = [np.nextafter(near, np.float32(-9), dtype=np.float32), near,
             np.nextafter(near, np.float32(9), dtype=np.float32), np.float32(3.0)]
    nll = np.array(steps + [0, 0, 0, 400, 400], dtype=np.float32)
    olds = np.array([old] * 4 + [500] * 3 + [0, 0], dtype=np.float32)
    adv = np.array([1, 1, 1, 0, 1, 0, -1, 1, -1], dtype=np.float32)
    d = cu_dev(nll, olds, adv)
    got = ah.policy_loss(*d, clip_low=0.25, clip_high=0.25, reduction="sum")
    ah.check()
    g = got["dnll"].cpu().double().numpy()
    for n in range(3):  # FP32 inputs decide exactly which side of the border they lie on
        inside = float(old) - float(nll[n]) <= x
        want = np.exp(float(old) - float(nll[n])) if inside else 0.0
        assert abs(g[n] - want) <= 16 * U * 1.3, n
    assert list(g[3:6]) == [0, 0, 0] and g[6] == -np.inf and g[7] == 0 and g[8] == 0
    s = got["stats"].cpu().numpy()
    assert s[0] == np.inf and s[3] == sum(float(old) - float(v) > x for v in nll[:3]) + 2


@pytest.mark.gpu
@pytest.mark.parametrize("reduction", ["token", "sequence", "sum"])
def test_policy_all_masked_and_no_tokens(cuda_ok, reduction):
    cu = torch.tensor([0, 0, 4], dtype=torch.int32, device="cuda")
    nan = torch.full((7,), float("nan"), device="cuda")
    w = torch.zeros(7, device="cuda")
    got = ah.policy_loss(nan, nan, nan, nll_ref=nan, weights=w, cu_seqlens=cu, kl_coef=1.0,
                         reduction=reduction)
    none = ah.policy_loss(nan[:0], nan[:0], nan[:0], cu_seqlens=cu[:1], reduction=reduction)
    ah.check()
    assert got["dnll"].tolist() == [0] * 7 and got["stats"].tolist() == [0] * 4
    assert none["dnll"].numel() == 0 and none["stats"].tolist() == [0] * 4


@pytest.mark.gpu
@pytest.mark.parametrize("reduction", ["token", "sequence", "sum"])
def test_tokens_outside_every_sequence_are_masked(cuda_ok, reduction):
    nll, old, ref, w, rng = make_tokens(700, 3)
    cu = np.array([5, 5, 300, 301], dtype=np.int32)
    adv = rng.normal(size=700).astype(np.float32)
    want = policy_ref(nll, old, adv, ref, w, cu, reduction=reduction, beta=0.5)
    for a in (nll, old, ref, adv):
        a[:5] = np.nan
        a[301:] = np.nan
    d = cu_dev(nll, old, adv, ref, w, cu)
    got = ah.policy_loss(d[0], d[1], d[2], nll_ref=d[3], weights=d[4], cu_seqlens=d[5], kl_coef=0.5,
                         reduction=reduction)
    pref = ah.preference_loss(d[0], d[5], torch.tensor([[1, 2]], dtype=torch.int32, device="cuda"),
                              nll_ref=d[3], weights=d[4])
    ah.check()
    close(got["dnll"], want["dnll"], U * (want["size"] + np.abs(want["dnll"])), "dnll")
    g = pref["dnll"].cpu().numpy()
    assert np.isfinite(g).all() and not g[:5].any() and not g[301:].any() and g[5:301].any()


def test_policy_reference_gradient_is_that_of_its_loss():
    """The FP64 formula's gradient against central differences (no token near a clip border)."""
    nll, old, ref, w, rng = make_tokens(40, 8)
    cu = offsets([7, 0, 20, 13])
    adv = rng.normal(size=40).astype(np.float32)
    x = nll.astype(np.float64)
    for reduction in ("token", "sequence", "sum"):
        args = (old, adv, ref, w, cu)
        g = policy_ref(x, *args, beta=0.3, reduction=reduction)["dnll"]
        for n in range(0, 40, 3):
            h = 1e-6
            lo, hi = x.copy(), x.copy()
            lo[n] -= h
            hi[n] += h
            d = (policy_ref(hi, *args, beta=0.3, reduction=reduction)["stats"][0]
                 - policy_ref(lo, *args, beta=0.3, reduction=reduction)["stats"][0]) / (2 * h)
            assert abs(d - g[n]) <= 1e-7 + 1e-6 * abs(g[n])


# ---- preference loss --------------------------------------------------------------------
def make_pairs(B, P, rng):
    return rng.integers(0, B, size=(P, 2)).astype(np.int32)


@pytest.mark.gpu
@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "ipo"])
@pytest.mark.parametrize("average", [False, True])
def test_preference_loss_matches_formula(cuda_ok, lens, kind, average):
    cu = offsets(LENS[lens])
    N, B = int(cu[-1]), len(cu) - 1
    nll, _, ref, w, rng = make_tokens(N, 21, spread=0.1)
    pairs = make_pairs(B, 37 if B < 100 else 3000, rng)
    if kind == "hinge":
        ref = None
    if kind == "ipo":
        w = None
    smooth = 0.1 if kind == "sigmoid" else 0.0
    want = preference_ref(nll, cu, pairs, ref, w, 0.2, kind, smooth, 0.05, average)
    if w is not None:
        nll[w == 0] = np.nan
    d = cu_dev(nll, cu, pairs, ref, w)
    got = ah.preference_loss(d[0], d[1], d[2], nll_ref=d[3], weights=d[4], beta=0.2, kind=kind,
                             label_smoothing=smooth, margin=0.05, average=average)
    ah.check()
    # everything is FP64 and rounded once: half a step, and what FP64 sums of this size lose
    slip = 1e-12
    close(got["dnll"], want["dnll"], U * np.abs(want["dnll"]) + slip * (want["size"] + 1e-30), "dnll")
    for k in ("pair_loss", "rewards", "loss"):
        close(got[k], want[k], 1.001 * U * np.abs(want[k]) + slip * (1 + np.abs(want[k])), k)


@pytest.mark.gpu
def test_preference_same_sequence_in_many_pairs(cuda_ok):
    """One answer on both sides of many pairs, a pair of an answer with itself, tiny slopes next
    to large ones: integer sums lose nothing and their order does not matter."""
    cu = offsets([400, 3, 50, 1])
    nll, _, ref, w, rng = make_tokens(int(cu[-1]), 2, spread=2.0)
    pairs = np.array([[0, 1], [2, 0]] * 2500 + [[0, 0], [3, 3], [1, 3]], dtype=np.int32)
    want = preference_ref(nll, cu, pairs, ref, w, 0.5)
    d = cu_dev(nll, cu, pairs, ref, w)
    a = ah.preference_loss(d[0], d[1], d[2], nll_ref=d[3], weights=d[4], beta=0.5)
    close(a["dnll"], want["dnll"], U * np.abs(want["dnll"]) + 1e-12 * want["size"], "dnll")
    for _ in range(3):
        b = ah.preference_loss(d[0], d[1], d[2], nll_ref=d[3], weights=d[4], beta=0.5)
        assert all(torch.equal(a[k], b[k]) for k in a)
    ah.check()


@pytest.mark.gpu
def test_preference_extremes(cuda_ok):
    """Margins that overflow exp either way, and no pairs at all."""
    cu = offsets([1, 1, 1])
    nll = np.array([0.0, 5e4, 3.0], dtype=np.float32)
    pairs = np.array([[0, 1], [1, 0], [2, 2]], dtype=np.int32)
    d = cu_dev(nll, cu, pairs)
    got = ah.preference_loss(*d, beta=1.0)
    none = ah.preference_loss(d[0], d[1], d[2][:0])
    empty = ah.preference_loss(d[0][:0], torch.zeros(4, dtype=torch.int32, device="cuda"), d[2])
    ah.check()
    close(got["pair_loss"], np.array([0.0, 5e4, np.log(2)]), 5e4 * U * np.array([0, 1, 1e-4]), "pair")
    # the second pair's loss is nll[1] - nll[0]; the others are flat or cancel
    close(got["dnll"], np.array([-1.0, 1.0, 0.0]) / 3, U, "dnll")
    assert none["loss"].tolist() == [0] and none["dnll"].tolist() == [0] * 3
    close(empty["loss"], np.array([np.log(2)]), U, "empty sequences")


@pytest.mark.gpu
def test_bad_pairs_and_offsets_are_reported(cuda_ok):
    nll, old, ref, w, rng = make_tokens(1000, 4)
    cu = offsets([400, 600])
    adv = rng.normal(size=1000).astype(np.float32)
    d = cu_dev(nll, old, adv, cu)
    for pairs in ([[0, 2], [0, 1]], [[-1, 0], [0, 1]], [[2 ** 31 - 1, 0], [0, 1]]):
        p = torch.tensor(pairs, dtype=torch.int64).to(torch.int32).cuda()
        got = ah.preference_loss(d[0], d[3], p)
        with pytest.raises(ah.ArcheadError) as e:
            ah.check()
        assert e.value.status == E["ARCHEAD_ERR_SEGMENT"]
        pl = got["pair_loss"].cpu().numpy()
        assert np.isnan(pl[0]) and np.isfinite(pl[1]) and torch.isnan(got["loss"]).all()
        assert torch.isfinite(got["dnll"]).all()
    for bad in ([0, 700, 400], [-5, 10, 1000], [0, 400, 1001], [0, 2 ** 31 - 1, -2 ** 31]):
        c = torch.tensor(bad, dtype=torch.int64).to(torch.int32).cuda()
        for reduction in ("token", "sequence", "sum"):
            for weights in (None, torch.ones(1000, device="cuda")):
                ah.policy_loss(d[0], d[1], d[2][:2].contiguous(), cu_seqlens=c, per_sequence=True,
                               weights=weights, reduction=reduction)
                with pytest.raises(ah.ArcheadError):
                    ah.check()
        ah.preference_loss(d[0], c, torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"))
        with pytest.raises(ah.ArcheadError):
            ah.check()
    ah.check()


@pytest.mark.gpu
@pytest.mark.parametrize("lens", ["many short", "one long", "many"])
def test_losses_repeat_bit_for_bit_and_under_a_graph(cuda_ok, lens):
    cu = offsets(LENS[lens])
    N, B = int(cu[-1]), len(cu) - 1
    nll, old, ref, w, rng = make_tokens(N, 6)
    adv = rng.normal(size=B).astype(np.float32)
    pairs = make_pairs(B, 500, rng)
    d = cu_dev(nll, old, adv, ref, w, cu, pairs)

    def both():
        a = ah.policy_loss(d[0], d[1], d[2], nll_ref=d[3], weights=d[4], cu_seqlens=d[5],
                           per_sequence=True, kl_coef=0.1, reduction="sequence")
        return [*a.values(), *ah.preference_loss(d[0], d[5], d[6], nll_ref=d[3], weights=d[4]).values()]

    first = [t.clone() for t in both()]
    assert all(torch.equal(a, b) for a, b in zip(first, both()))
    side = torch.cuda.Stream()
    graphs = []
    for _ in range(2):  # two graphs of the same work live at once
        g = torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=side):
            out = both()
        graphs.append((g, out))
    d[0].copy_(torch.from_numpy(old).cuda())  # new inputs in the captured places
    want = both()
    for g, out in graphs:
        g.replay()
    torch.cuda.synchronize()
    for g, out in graphs:
        assert all(torch.equal(a, b) for a, b in zip(want, out))
    assert not torch.equal(first[1], want[1])
    ah.check()


@pytest.mark.gpu
@pytest.mark.parametrize("lens", ["piece edges", "many", "one long"])
def test_arrays_aligned_to_four_bytes_only(cuda_ok, lens):
    """The same values at an address that is no multiple of 16 give the same bits."""
    cu = offsets(LENS[lens])
    N, B = int(cu[-1]), len(cu) - 1
    nll, old, ref, w, rng = make_tokens(N, 14)
    adv = rng.normal(size=N).astype(np.float32)
    d = cu_dev(nll, old, adv, ref, w, cu, make_pairs(B, 40, rng))

    def moved(t):
        b = torch.empty(t.numel() + 1, device="cuda")
        b[1:] = t
        assert b[1:].data_ptr() % 16 == 4
        return b[1:]

    def both(nll, old, adv, ref, w):
        a = ah.policy_loss(nll, old, adv, nll_ref=ref, weights=w, cu_seqlens=d[5], kl_coef=0.1,
                           reduction="sequence")
        return [*a.values(), *ah.preference_loss(nll, d[5], d[6], nll_ref=ref, weights=w).values()]

    for a, b in zip(both(*d[:5]), both(*[moved(t) for t in d[:5]])):
        assert torch.equal(a, b)
    ah.check()


@pytest.mark.gpu
@pytest.mark.parametrize("B", [600, 3000])
def test_many_sequences_of_few_tokens(cuda_ok, B):
    """More sequences than tokens, most of them empty, many at one place."""
    rng = np.random.default_rng(B)
    lens = np.where(rng.random(B) < 0.9, 0, rng.integers(1, 4, size=B))
    lens[100:400] = 0
    cu = offsets(lens)
    N = int(cu[-1])
    nll, old, ref, w, rng = make_tokens(N, 15)
    adv = rng.normal(size=B).astype(np.float32)
    want = policy_ref(nll, old, adv, ref, w, cu, True, reduction="sequence", beta=0.1)
    pairs = make_pairs(B, 2000, rng)
    wantp = preference_ref(nll, cu, pairs, ref, w, 0.3, average=True)
    d = cu_dev(nll, old, adv, ref, w, cu, pairs)
    got = ah.policy_loss(d[0], d[1], d[2], nll_ref=d[3], weights=d[4], cu_seqlens=d[5],
                         per_sequence=True, kl_coef=0.1, reduction="sequence")
    gotp = ah.preference_loss(d[0], d[5], d[6], nll_ref=d[3], weights=d[4], beta=0.3, average=True)
    ah.check()
    close(got["dnll"], want["dnll"], U * (want["size"] + np.abs(want["dnll"])), "policy")
    close(gotp["dnll"], wantp["dnll"], U * np.abs(wantp["dnll"]) + 1e-12 * wantp["size"], "preference")


# ---- refusals (host) --------------------------------------------------------------------
@pytest.fixture(scope="module")
def L():
    if not os.path.exists(_lib.LIB_PATH):
        from packed_int4_lm_b200 import build
        build.build()
    return _lib.lib()


def test_loss_argument_errors(L):
    a = 0x1000000

    def policy(nll=a, old=a, ref=None, adv=a, w=None, cu=None, dnll=a, stats=a, N=8, B=0, per=0,
               lo=0.2, hi=0.2, beta=0.0, red=0):
        return L.archead_policy_loss(nll, old, ref, adv, w, cu, dnll, stats, N, B, per, lo, hi, beta,
                                     red, None)

    for kw, code in (
            (dict(nll=None), "NULLPTR"), (dict(old=None), "NULLPTR"), (dict(adv=None), "NULLPTR"),
            (dict(dnll=None), "NULLPTR"), (dict(stats=None), "NULLPTR"),
            (dict(per=1), "NULLPTR"), (dict(red=1), "NULLPTR"),
            (dict(nll=a + 2), "ALIGN"), (dict(w=a + 1), "ALIGN"), (dict(cu=a + 2, B=1), "ALIGN"),
            (dict(N=-1), "SHAPE"), (dict(N=1 << 31), "SHAPE"), (dict(B=-1), "SHAPE"),
            (dict(B=(1 << 31) - 1), "SHAPE"), (dict(red=3), "SHAPE"), (dict(red=-1), "SHAPE"),
            (dict(lo=1.0), "SHAPE"), (dict(lo=-0.1), "SHAPE"), (dict(hi=-0.1), "SHAPE"),
            (dict(hi=float("inf")), "SHAPE"), (dict(lo=float("nan")), "SHAPE"),
            (dict(beta=float("nan")), "SHAPE")):
        assert policy(**kw) == E["ARCHEAD_ERR_" + code], kw

    def pref(nll=a, ref=None, w=None, cu=a, pairs=a, dnll=a, loss=a, pl=a, rw=a, N=8, B=2, P=1,
             kind=0, avg=0, beta=0.1, smooth=0.0, margin=0.0):
        return L.archead_preference_loss(nll, ref, w, cu, pairs, dnll, loss, pl, rw, N, B, P, kind,
                                         avg, beta, smooth, margin, None)

    for kw, code in (
            (dict(nll=None), "NULLPTR"), (dict(cu=None), "NULLPTR"), (dict(pairs=None), "NULLPTR"),
            (dict(loss=None), "NULLPTR"), (dict(pl=None), "NULLPTR"), (dict(rw=None), "NULLPTR"),
            (dict(dnll=None), "NULLPTR"), (dict(pairs=a + 2), "ALIGN"), (dict(rw=a + 1), "ALIGN"),
            (dict(P=-1), "SHAPE"), (dict(kind=3), "SHAPE"), (dict(beta=0.0), "SHAPE"),
            (dict(beta=float("inf")), "SHAPE"), (dict(smooth=1.0), "SHAPE"),
            (dict(kind=1, smooth=0.1), "SHAPE"), (dict(margin=float("nan")), "SHAPE"),
            (dict(N=1 << 31), "SHAPE")):
        assert pref(**kw) == E["ARCHEAD_ERR_" + code], kw


def test_loss_binding_refuses_what_it_cannot_take():
    x = torch.zeros(4)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        ah.policy_loss(x, x, x)  # not on a GPU
    with pytest.raises(ValueError):
        ah.policy_loss(x, x, x, reduction="mean")
    with pytest.raises(ValueError):
        ah.preference_loss(x, i, torch.zeros(1, 2, dtype=torch.int32), kind="other")
    with pytest.raises(ValueError):
        ah.preference_loss(x, None, torch.zeros(1, 2, dtype=torch.int32))


@pytest.mark.gpu
def test_loss_binding_checks_shapes_and_types(cuda_ok):
    x = torch.zeros(6, device="cuda")
    cu = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    pairs = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    for bad in (x.double(), x[:5], x.cpu(), torch.zeros(12, device="cuda")[::2], x[None]):
        for kw in ("nll_old", "advantages"):
            args = {"nll_old": x, "advantages": x, kw: bad}
            with pytest.raises(ValueError):
                ah.policy_loss(x, args["nll_old"], args["advantages"])
        with pytest.raises(ValueError):
            ah.preference_loss(x, cu, pairs, weights=bad)
    with pytest.raises(ValueError):
        ah.policy_loss(x, x, x, reduction="sequence")
    with pytest.raises(ValueError):
        ah.policy_loss(x, x, x, per_sequence=True)
    with pytest.raises(ValueError):
        ah.preference_loss(x, cu.long(), pairs)
    with pytest.raises(ValueError):
        ah.preference_loss(x, cu, pairs.view(2))
