"""The losses on per-token NLLs at the ends of their range: infinities and NaN, slopes of very
different size, cancelling sums, both ends of the one-block form, the largest sizes and other
streams.  Formulas and tolerances as in test_losses.py."""
import numpy as np
import pytest
import torch

import packed_int4_lm_b200 as ah
from test_losses import U, close, cu_dev, make_pairs, make_tokens, offsets, policy_ref, preference_ref

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("border", [False, True])
def test_policy_nan_advantage_is_nan_on_every_side_of_the_border(cuda_ok, border):
    """A token whose advantage is NaN gets NaN wherever its ratio lies, and is not clipped, whether
    or not a token beside it lies on the clip border; no other token changes."""
    nll, old, ref, w, rng = make_tokens(300, 31)
    x = rng.choice([-2.0, -0.1, 0.1, 2.0], size=300)
    old = (nll + x).astype(np.float32)
    adv = rng.normal(size=300).astype(np.float32)
    if border:
        nll[::64], old[::64], adv[::64] = 0, np.float32(np.log1p(0.2)), 1
    bad = np.arange(300) % 7 == 3
    assert (x[bad] == -2.0).any() and (x[bad] == 2.0).any()
    d = cu_dev(nll, old, adv, np.where(bad, np.float32(np.nan), adv), (~bad).astype(np.float32))
    kw = dict(clip_low=0.2, clip_high=0.2, reduction="sum")
    want = ah.policy_loss(d[0], d[1], d[2], weights=d[4], **kw)
    got = ah.policy_loss(d[0], d[1], d[3], **kw)
    ah.check()
    g, b = got["dnll"].cpu().numpy(), want["dnll"].cpu().numpy()
    assert np.isnan(g[bad]).all()
    assert (g[~bad] == b[~bad]).all()
    assert torch.isnan(got["stats"][:2]).all() and got["stats"][3] == want["stats"][3]


def test_policy_advantage_zero_keeps_a_nan(cuda_ok):
    """Advantage 0 times an infinite ratio is 0; a NaN log-probability stays NaN."""
    nll = np.array([NAN, 1, 0, -np.inf, 2], dtype=np.float32)
    old = np.array([1, NAN, 500, 1, 2], dtype=np.float32)
    d = cu_dev(nll, old, np.zeros(5, dtype=np.float32))
    got = ah.policy_loss(*d, reduction="sum")
    ah.check()
    g = got["dnll"].cpu().numpy()
    assert np.isnan(g[:2]).all() and not g[2:].any()
    assert torch.isnan(got["stats"][:2]).all()
    good = ah.policy_loss(*[t[2:].contiguous() for t in d], reduction="sum")
    ah.check()
    assert good["stats"].tolist() == [0] * 4


def test_policy_infinite_reference(cuda_ok):
    """nll_ref = +inf: z = -inf, the KL term e^z - z - 1 is infinite and its derivative e^z - 1 is -1.
    Far below 0 the derivative keeps its precision."""
    nll, old, ref, w, rng = make_tokens(40, 32)
    adv = rng.normal(size=40).astype(np.float32)
    ref[5] = np.inf
    ref[6:12] = nll[6:12] + np.array([1.5, 4, 20, 90, 1e4, 3e38], dtype=np.float32)
    d = cu_dev(nll, old, adv, ref)
    got = ah.policy_loss(d[0], d[1], d[2], nll_ref=d[3], kl_coef=0.5, reduction="sum", clip_low=0.9, clip_high=9)
    ah.check()
    r = np.exp(old.astype(np.float64) - nll)
    z = nll.astype(np.float64) - ref
    want = r * adv + 0.5 * np.expm1(z)
    # half steps: |z| of the difference inside exp times e^z, a few of exp and the products
    size = (np.abs(old.astype(np.float64) - nll) + 8) * r * np.abs(adv) + 0.5 * ((np.minimum(np.abs(z), 1e3) + 8) * np.exp(z) + 4)
    close(got["dnll"], want, U * (size + np.abs(want)), "dnll")
    s = got["stats"].cpu().numpy()
    assert s[0] == np.inf and s[2] == np.inf and np.isfinite(s[1])


def test_policy_far_ratios_keep_their_precision(cuda_ok):
    """Ratios and KL terms of large and tiny differences, which are exact here."""
    x = np.array([-100, -87, -60, -31.5, -8, -1, 1, 8, 31.5, 60, 87], dtype=np.float32)
    adv = np.where(x > 0, -1, 1).astype(np.float32)  # (the clipped side is never the smaller one)
    zero = np.zeros_like(x)
    d = cu_dev(zero, x, adv, -x)
    got = ah.policy_loss(d[0], d[1], d[2], reduction="sum")
    kl = ah.policy_loss(d[0], d[0], torch.zeros_like(d[0]), nll_ref=d[3], kl_coef=1.0, reduction="sum")
    ah.check()
    r = np.exp(x.astype(np.float64)) * adv
    # an exponential within two units in the last place (four half steps), a product
    close(got["dnll"], r, 6 * U * np.abs(r) + 2.0 ** -149, "dnll")
    want = np.expm1(x.astype(np.float64))
    close(kl["dnll"], want, 6 * U * (np.abs(want) + 1), "kl")


def test_policy_reference_without_a_coefficient_leaves_the_gradient(cuda_ok):
    """With kl_coef = 0 the reference is only reported: the loss and its gradient are the
    surrogate's, whatever the KL term is."""
    nll, old, ref, w, rng = make_tokens(600, 33)
    adv = rng.normal(size=600).astype(np.float32)
    ref[::3] = (nll - rng.choice([100, 89, 1e30], size=600).astype(np.float32))[::3]
    ref[1::7] = rng.choice([np.nan, np.inf, -np.inf], size=600)[1::7]
    d = cu_dev(nll, old, adv, ref)
    for reduction in ("sum", "token"):
        want = ah.policy_loss(d[0], d[1], d[2], reduction=reduction)
        got = ah.policy_loss(d[0], d[1], d[2], nll_ref=d[3], kl_coef=0.0, reduction=reduction)
        ah.check()
        assert torch.equal(got["dnll"], want["dnll"])
        assert torch.equal(got["stats"][[0, 1, 3]], want["stats"][[0, 1, 3]])


@pytest.mark.parametrize("N", [512, 40000])
def test_policy_sums_of_cancelling_tokens(cuda_ok, N):
    """Equal log-probabilities make every share -A: large ones that cancel leave the small ones,
    exactly, as these sums are exact in FP64."""
    rng = np.random.default_rng(N)
    at = np.arange(0, N, 4)
    for big in (2.0 ** 31, 3e38):
        adv = rng.integers(-9, 10, size=N).astype(np.float32)
        if big < 1e38:  # big, small, -big, small
            adv[at], adv[at + 2] = big, -big
            small = -(adv[at + 1].astype(np.float64).sum() + adv[at + 3].sum())
        else:  # what four tokens add up to passes FP32 in between
            adv[at], adv[at + 1], adv[at + 2], adv[at + 3] = big, big, -big, -big
            small = 0.0
        x = torch.ones(N, device="cuda")
        got = ah.policy_loss(x, x, torch.from_numpy(adv).cuda(), reduction="sum")
        ah.check()
        assert got["stats"].tolist() == [small, small, 0, 0]
        assert torch.equal(got["dnll"], torch.from_numpy(adv).cuda())


def test_preference_infinite_margin(cuda_ok):
    """A preferred answer that the reference gives probability 0: the loss without smoothing is 0
    and flat; with smoothing it is infinite."""
    nll = np.array([1, 2, 3], dtype=np.float32)
    ref = np.array([np.inf, 2, 1], dtype=np.float32)
    pairs = np.array([[0, 1], [2, 1]], dtype=np.int32)
    d = cu_dev(nll, offsets([1, 1, 1]), pairs, ref)
    got = ah.preference_loss(d[0], d[1], d[2], nll_ref=d[3], beta=0.5)
    other = ah.preference_loss(d[0], d[1], d[2], nll_ref=d[3], beta=0.5, label_smoothing=0.1)
    back = ah.preference_loss(d[0], d[1], d[2].flip(1).contiguous(), nll_ref=d[3], beta=0.5)
    ah.check()
    m = 0.5 * (-2.0 - 0.0)
    close(got["pair_loss"], np.array([0.0, np.log1p(np.exp(-m))]), 4 * U, "pair_loss")
    close(got["dnll"], np.array([0.0, -0.25, 0.25]) / (1 + np.exp(m)), 4 * U, "dnll")
    assert torch.isfinite(got["loss"]).all()
    assert other["pair_loss"][0] == INF and torch.isfinite(other["dnll"]).all()
    assert back["pair_loss"][0] == INF and back["dnll"][0] == -0.25


@pytest.mark.parametrize("copies", [1, 40])
@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "ipo"])
def test_preference_slopes_of_every_size(cuda_ok, kind, copies):
    """Pairs that are long decided, whose slopes fade as e^-m, beside fresh ones, and squared gaps of
    any size: every slope is right to its last bit, in one block and in the chain."""
    gaps = np.array([0.0, 1, 20, 50, 55, 60, 70, 80, 87, 100, 103, -30, -1000])
    if kind == "ipo":
        gaps = np.concatenate([gaps, [2e9, 3e9, 5e15, -7e20, 1e30, -1e37]])
    nll = np.zeros(2 * len(gaps), dtype=np.float32)
    nll[1::2] = gaps
    gaps = nll[1::2].astype(np.float64)
    nll, gaps = np.tile(nll, copies), np.tile(gaps, copies)
    P = len(gaps)
    pairs = np.arange(2 * P, dtype=np.int32).reshape(P, 2)
    d = cu_dev(nll, offsets([1] * (2 * P)), pairs)
    got = ah.preference_loss(*d, beta=1.0, kind=kind)
    assert (ah.last_launches() == 1) == (copies == 1)
    ah.check()
    if kind == "sigmoid":
        slope = -1 / (1 + np.exp(gaps))
    elif kind == "hinge":
        slope = np.where(gaps < 1, -1.0, 0.0)
    else:
        slope = 2 * (gaps - 0.5)
    want = np.stack([-slope, slope], 1).ravel() / P
    # FP64 rounded once: half a step, of the smallest FP32 number at least
    close(got["dnll"], want, 1.001 * U * np.abs(want) + 1.001 * 2.0 ** -150, kind)


def test_preference_slopes_past_every_size_are_nan(cuda_ok):
    """An infinite gap under the squared loss, and one whose slope passes what sums can hold, make
    the two answers' gradients NaN and no other's."""
    nll = np.array([0, np.inf, 0, 3e38, 0, 5], dtype=np.float32)
    w = np.array([1, 1, 1, 3e38, 1, 1], dtype=np.float32)
    d = cu_dev(nll, offsets([1] * 6), np.arange(6, dtype=np.int32).reshape(3, 2), w)
    got = ah.preference_loss(d[0], d[1], d[2], weights=d[3], kind="ipo", beta=1.0)
    ah.check()
    g = got["dnll"].cpu().numpy()
    assert np.isnan(g[:4]).all() and list(g[4:]) == [-3.0, 3.0]


@pytest.mark.parametrize("B", [33, 129, 255, 256, 257])
@pytest.mark.parametrize("reduction", ["token", "sequence", "sum"])
@pytest.mark.parametrize("per_seq", [False, True])
def test_policy_of_many_sequences_in_one_block(cuda_ok, B, reduction, per_seq):
    """Up to 256 sequences run in one launch, whose walk reloads its window of 32 and whose sums
    take two rounds of 128."""
    rng = np.random.default_rng(B)
    lens = rng.choice([0, 1, 2, 5, 33, 70], size=B)
    lens[B // 2:B // 2 + 20] = rng.integers(33, 60, size=20 if B > 50 else B - B // 2)[:20]
    cu = offsets(lens)
    N = int(cu[-1])
    assert N <= 32 * 256
    nll, old, ref, w, rng = make_tokens(N, 41)
    w[cu[3]:cu[9]] = 0
    adv = rng.normal(size=B if per_seq else N).astype(np.float32)
    kw = dict(lo=0.2, hi=0.3, beta=0.1, reduction=reduction)
    for weights in (w, None):
        want = policy_ref(nll, old, adv, ref, weights, cu, per_seq, **kw)
        d = cu_dev(nll, old, adv, ref, weights, cu)
        got = ah.policy_loss(d[0], d[1], d[2], nll_ref=d[3], weights=d[4], cu_seqlens=d[5], per_sequence=per_seq,
                             clip_low=0.2, clip_high=0.3, kl_coef=0.1, reduction=reduction)
        assert (ah.last_launches() == 1) == (B <= 256)
        ah.check()
        close(got["dnll"], want["dnll"], U * (want["size"] + np.abs(want["dnll"])), "dnll")
        close(got["stats"], want["stats"], 2 * U * (want["mag"] + np.abs(want["stats"])), "stats")


@pytest.mark.parametrize("B,P", [(33, 64), (129, 65), (255, 192), (256, 192), (256, 193), (257, 65)])
@pytest.mark.parametrize("average", [False, True])
def test_preference_of_many_sequences_in_one_block(cuda_ok, B, P, average):
    """Up to 256 sequences and 192 pairs run in one launch, 64 pairs a round."""
    rng = np.random.default_rng(B + P)
    cu = offsets(rng.choice([0, 1, 2, 5, 33, 70], size=B))
    N = int(cu[-1])
    nll, _, ref, w, rng = make_tokens(N, 42, spread=0.1)
    pairs = make_pairs(B, P, rng)
    want = preference_ref(nll, cu, pairs, ref, w, 0.2, "sigmoid", 0.1, 0.05, average)
    d = cu_dev(nll, cu, pairs, ref, w)
    got = ah.preference_loss(d[0], d[1], d[2], nll_ref=d[3], weights=d[4], beta=0.2, label_smoothing=0.1, margin=0.05,
                             average=average)
    assert (ah.last_launches() == 1) == (B <= 256 and P <= 192)
    ah.check()
    slip = 1e-12
    close(got["dnll"], want["dnll"], U * np.abs(want["dnll"]) + slip * (want["size"] + 1e-30), "dnll")
    for k in ("pair_loss", "rewards", "loss"):
        close(got[k], want[k], 1.001 * U * np.abs(want[k]) + slip * (1 + np.abs(want[k])), k)


def test_preference_average_of_long_sequences(cuda_ok):
    """Sequences of millions of tokens beside short ones: a sequence's weight is the same in every
    piece of it."""
    lens = [3, 5_000_000, 40, 3_000_001, 0, 2]
    cu = offsets(lens)
    N = int(cu[-1])
    rng = np.random.default_rng(7)
    nll = np.abs(rng.normal(size=N)).astype(np.float32)
    w = rng.choice([0.0, 1.0, 0.5], size=N).astype(np.float32)
    pairs = np.array([[1, 3], [0, 1], [3, 5], [2, 4]], dtype=np.int32)
    want = preference_ref(nll, cu, pairs, None, w, 0.7, average=True)
    d = cu_dev(nll, cu, pairs, w)
    got = ah.preference_loss(d[0], d[1], d[2], weights=d[3], beta=0.7, average=True)
    ah.check()
    close(got["dnll"], want["dnll"], U * np.abs(want["dnll"]) + 1e-12 * want["size"], "dnll")
    close(got["rewards"], want["rewards"], 1.001 * U * np.abs(want["rewards"]) + 1e-12, "rewards")


def _largest(fill):
    """A float array of the largest size, filled a slice at a time."""
    N = 2 ** 31 - 1
    x = torch.empty(N, device="cuda")
    for n0 in range(0, N, 1 << 28):
        n1 = min(N, n0 + (1 << 28))
        x[n0:n1] = fill(torch.arange(n0, n1, device="cuda", dtype=torch.int64))
    return x, N


@pytest.mark.parametrize("average", [False, True])
def test_losses_of_the_most_tokens(cuda_ok, average):
    """2^31 - 1 tokens: one long sequence and five of one token behind it, whose last offsets are the
    largest 32-bit number.  The values are multiples of 2^-10, so every sum is exact."""
    nll, N = _largest(lambda i: ((i * 40503) & 1023).float() / 1024)
    cu = torch.tensor([0] + [N - 5 + k for k in range(6)], dtype=torch.int64).to(torch.int32).cuda()
    w = torch.ones(N, device="cuda")
    parts = [slice(n0, min(N, n0 + (1 << 28))) for n0 in range(0, N, 1 << 28)]
    last = nll[-5:].double().cpu().numpy()
    total = sum(nll[p].double().sum().item() for p in parts) - last.sum()
    pairs = torch.tensor([[0, 1], [2, 3], [4, 5], [5, 0]], dtype=torch.int32, device="cuda")
    f = np.concatenate([[-total / (N - 5) if average else -total], -last])
    beta = 1.0 if average else 2.0 ** -30
    a, b = pairs.cpu().numpy().T
    m = beta * (f[a] - f[b])
    back = np.zeros(6)
    np.add.at(back, a, -beta / (1 + np.exp(m)) / 4)
    np.add.at(back, b, beta / (1 + np.exp(m)) / 4)
    first = -back[0] / (N - 5 if average else 1)
    for weights in (None, w):
        got = ah.preference_loss(nll, cu, pairs, weights=weights, beta=beta, average=average)
        ah.check()
        for k, want in (("pair_loss", np.logaddexp(0, -m)), ("rewards", beta * np.stack([f[a], f[b]], 1))):
            close(got[k], want, 1.001 * U * np.abs(want) + 1e-12, k)
        g = got["dnll"]
        close(g[-5:], -back[1:], 1.001 * U * np.abs(back[1:]) + 1e-12 * beta, "dnll")
        for p in parts:
            part = g[p.start:min(p.stop, N - 5)]
            assert max(abs(part.min().item() - first), abs(part.max().item() - first)) <= 1.001 * U * abs(first)
        del got, g, part
    adv = torch.tensor([0.5, 1, -1, 2, -2, 3], device="cuda")
    got = ah.policy_loss(nll, nll, adv, weights=w, cu_seqlens=cu, per_sequence=True, reduction="sequence")
    ah.check()
    g = got["dnll"]
    close(g[-5:], np.array([1, -1, 2, -2, 3]) / 6, 4 * U, "policy dnll")
    want = 0.5 / 6 / (N - 5)
    assert abs(g[0].item() - want) <= 4 * U * want and abs(g[N - 6].item() - want) <= 4 * U * want
    close(got["stats"], np.array([-3.5 / 6, -3.5 / 6, 0, 0]), 1e-6, "stats")
    del got, g, nll, w
    torch.cuda.empty_cache()


def test_policy_of_the_most_sequences(cuda_ok):
    """2^31 - 2 sequences, all empty but the last ones: what those ten alone give."""
    B, N = 2 ** 31 - 2, 1000
    nll, old, ref, w, rng = make_tokens(N, 51)
    lens = [100] * 8 + [1, 199]
    adv = rng.normal(size=N).astype(np.float32)
    d = cu_dev(nll, old, adv, ref, offsets(lens))
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[-11:] = d[4]
    want = ah.policy_loss(d[0], d[1], d[2], nll_ref=d[3], cu_seqlens=d[4], kl_coef=0.1, reduction="sequence")
    got = ah.policy_loss(d[0], d[1], d[2], nll_ref=d[3], cu_seqlens=cu, kl_coef=0.1, reduction="sequence")
    ah.check()
    assert torch.equal(got["dnll"], want["dnll"])
    close(got["stats"], want["stats"].cpu().double().numpy(), 2 * U * np.abs(want["stats"].cpu().double().numpy()) + 1e-9, "stats")
    del cu
    torch.cuda.empty_cache()


@pytest.mark.parametrize("which", ["policy", "preference", "nll_lse", "nll_grad", "logits_grad", "logits", "nll",
                                   "nll_partials", "nll_merge", "agreement", "dequant"])
def test_outputs_on_another_stream_are_not_the_current_streams_memory(cuda_ok, which):
    """A call on another stream while the current one still has work that writes a freed tensor of
    the outputs' size: the outputs do not lie there."""
    from test_head_grad import head_of, make_dY
    head, W, M = head_of("g64")
    dh = ah.DeviceHead.from_canonical(head, "cuda")
    N = 200
    nll, old, ref, w, rng = make_tokens(N, 61)
    d = cu_dev(nll, old, rng.normal(size=N).astype(np.float32), offsets([100, 100]), np.array([[0, 1]], dtype=np.int32))
    H = torch.from_numpy(rng.normal(size=(N, head["D"]))).to(torch.bfloat16).cuda()
    t = torch.from_numpy(rng.integers(0, head["V"], size=N).astype(np.int32)).cuda()
    nl, ls = ah.nll_lse(H, dh, t)
    dY = torch.from_numpy(make_dY(N, head["V"], 3)).cuda()
    t2, part = torch.stack([t, t], 1), ah.nll_partials(H, dh, t, 0, head["V"])
    side = torch.cuda.Stream()

    def call(stream=None):
        if which == "policy":
            return list(ah.policy_loss(d[0], d[1], d[2], stream=stream).values())
        if which == "preference":
            return list(ah.preference_loss(d[0], d[3], d[4], stream=stream).values())
        if which == "nll_lse":
            return list(ah.nll_lse(H, dh, t, stream=stream))
        if which == "nll_grad":
            return [ah.nll_grad(H, dh, t, nl, ls, d[2], stream=stream)]
        if which == "logits_grad":
            return [ah.logits_grad(dY, dh, stream=stream)]
        if which == "logits":
            return [ah.logits(H, dh, stream=stream)]
        if which == "nll":  # (a copy of the targets is made on the way)
            return [ah.nll(H, dh, t2[:, 0], stream=stream)]
        if which == "nll_partials":
            return [ah.nll_partials(H, dh, t2[:, 0], 0, head["V"], stream=stream)]
        if which == "nll_merge":
            return [ah.nll_merge(part[None], stream=stream)]
        if which == "agreement":
            return list(ah.agreement(H, dh, dY, stream=stream).values())
        return list(ah.dequant(dh, 128, 500, stream=stream).values())

    want = [o.clone() for o in call()]
    call(side)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # some 50 ms
    old_memory = [torch.empty_like(o) for o in want]
    for o in old_memory:
        o.fill_(-7)
    addresses = {o.data_ptr() for o in old_memory}
    del o, old_memory
    got = call(side)
    assert addresses.isdisjoint(o.data_ptr() for o in got)
    side.synchronize()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    ah.check()


@pytest.mark.parametrize("which", ["nll_lse", "nll_grad", "logits_grad"])
def test_a_head_that_is_dropped_after_a_call_on_another_stream(cuda_ok, which):
    """The head's memory is not handed out again while a stream that was given still reads it."""
    from test_head_grad import HEADS, make_dY
    head = HEADS["g64"]()
    N, V, D = 40, head["V"], head["D"]
    rng = np.random.default_rng(3)
    H = torch.from_numpy(rng.normal(size=(N, D))).to(torch.bfloat16).cuda()
    t = torch.from_numpy(rng.integers(0, V, size=N).astype(np.int32)).cuda()
    dn = torch.from_numpy(rng.normal(size=N).astype(np.float32)).cuda()
    dY = torch.from_numpy(make_dY(N, V, 3)).cuda()
    dh = ah.DeviceHead.from_canonical(head, "cuda")
    nl, ls = ah.nll_lse(H, dh, t)
    side = torch.cuda.Stream()

    def call(dh, stream=None):
        if which == "nll_lse":
            return list(ah.nll_lse(H, dh, t, stream=stream))
        if which == "nll_grad":
            return [ah.nll_grad(H, dh, t, nl, ls, dn, stream=stream)]
        return [ah.logits_grad(dY, dh, stream=stream)]

    want = [o.clone() for o in call(dh)]
    call(dh, side)
    torch.cuda.synchronize()
    shapes = [(x.shape, x.dtype) for x in dh.tensors.values()]
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    got = call(dh, side)
    used = {x.data_ptr() for x in dh.tensors.values()}
    del dh
    again = [torch.full(s, 1, dtype=d, device="cuda") for s, d in shapes]
    assert used.isdisjoint(x.data_ptr() for x in again)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    ah.check()
