"""The gradients on the paths that large batches take, at the ends of the heads' scales and with
NLLs from calls of another size.  Formulas and tolerances as in test_head_grad.py."""
import os
import re

import numpy as np
import pytest
import torch

import oracle
import packed_int4_lm_b200 as ah
from test_head_grad import BF16, PROD, close, head_of, magnitudes, make_dY, make_head, nll_tol, smallest_step
from workloads import bf16_bits, make_channel_scales, make_hidden, make_targets

pytestmark = pytest.mark.gpu


def wide_tiles():
    """Tiles of 256 tokens x 256 rows from which on the logits run in them."""
    api = os.path.join(os.path.dirname(ah.__file__), "csrc", "archead_api.cu")
    return int(re.search(r"kWideTiles = (\d+);", open(api).read()).group(1))


@pytest.mark.parametrize("name,N", [("g64", 19275), ("g32 odd", 15437), ("g128", 4700), ("g256 ranks 128", 19275),
                                    ("wide scales", 19275)])
def test_nll_grad_in_wide_tiles(cuda_ok, name, N):
    """Batches that fill the SMs twice with tiles of 256 tokens x 256 rows: several blocks of columns,
    ranks of every kind, a last tile of tokens without its second half.  240 of the tokens, the last
    ones among them, against FP64."""
    head, W, M = head_of(name)
    V, D = head["V"], head["D"]
    assert -(-V // 256) * -(-N // 256) >= wide_tiles() and -(-N // 128) % 2 == 1 and N % 128
    dh = ah.DeviceHead.from_canonical(head, "cuda")
    rng = np.random.default_rng(N)
    rows = np.unique(np.r_[rng.integers(0, N, size=160), N - 80:N])
    H = make_hidden(N, make_channel_scales(D, 0.5, 4, 20.0, 1), 2)
    tg = make_targets(N, V, 3).numpy()
    dnll = rng.normal(size=N).astype(np.float32)
    dnll[rows[::7]] = 0
    t, Hd, dn = torch.from_numpy(tg).cuda(), H.cuda(), torch.from_numpy(dnll).cuda()
    nl, ls = ah.nll_lse(Hd, dh, t)
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
    # The NLL is the difference of a log-sum-exp and a logit, FP32 numbers off by up to 4 half steps of
    # the largest logit each.  A target may lead by chance (logits reach 1000 under the wide scales: 1 - p =
    # 1.2e-7 where lse = 386 has a half step of 1.5e-5), and then that error is its whole entry p - 1.
    slip = 4 * 2.0 ** -24 * np.abs(Y).max(1)[:, None]
    tol = nll_tol(head, P, Y, M, dnll[rows], want) + np.abs(dnll[rows])[:, None] * 2 * slip * M[tg[rows]]
    close(got[torch.from_numpy(rows).cuda()], want, tol, name)


def scaled_factors(head, e):
    """The same head with its left factors 2^e larger and its right ones as much smaller."""
    out = dict(head)
    for a, b in (("Ac", "Bc"), ("Aw", "Bw")):
        out["s" + a] = (head["s" + a] * np.float32(2.0 ** e)).astype(np.float32)
        out["s" + b] = (head["s" + b] * np.float32(2.0 ** -e)).astype(np.float32)
    return out


@pytest.mark.parametrize("e", [-20, 12, 23, 27])
@pytest.mark.parametrize("N", [3, 40, 300])
def test_factors_scaled_against_each_other(cuda_ok, N, e):
    """Left factors far above or below the residual's scale, with right ones that make up for it:
    neither may be lost.  With k as in row_scale, the scales c 2^-k of the residual are exact up to k = 24
    and rounded to multiples of 2^-24 from there: off by 2^-25 each, times S' = S 2^k and the entry's |q|."""
    head = scaled_factors(make_head(1000, 512, 20, 12, 64, seed=9), e)
    S = oracle.bf16_bits_to_f64(head["r_super"])
    k = np.floor(np.log2(128 * np.maximum(head["sAc"], head["sAw"]))) - np.floor(np.log2(np.where(S > 0, S, 1))) - 13
    k[S == 0] = 0
    assert (k.max() <= 24) == (e < 27) and k.max() <= 28
    W, M = magnitudes(head)
    dh = ah.DeviceHead.from_canonical(head, "cuda")
    dY = make_dY(N, head["V"], 10 + N)
    got = ah.logits_grad(torch.from_numpy(dY).cuda(), dh)
    ah.check()
    size = np.abs(dY).astype(np.float64)
    codes = np.repeat(head["r_code"][:head["V"]].astype(np.float64) * S[:, None], head["g"], axis=1)
    q = np.divide(np.abs(oracle.unpack_residual(head)), codes, out=np.zeros((head["V"], head["D"])), where=codes > 0)
    fade = q * np.where(k > 24, 2.0 ** -25 * S * 2.0 ** k, 0)[:, None]
    want = dY.astype(np.float64) @ W
    close(got, want, BF16 * np.abs(want) + PROD * (size @ M) + smallest_step(head, M, dY) + size @ fade, e)


@pytest.mark.parametrize("name", ["g64", "g128"])
def test_nll_grad_with_nlls_of_smaller_batches(cuda_ok, name):
    """NLLs and log-sum-exps taken eight tokens at a time (another kernel, other rounding), the
    gradient of all tokens at once; confident tokens among them."""
    head, W, M = head_of(name)
    dh = ah.DeviceHead.from_canonical(head, "cuda")
    N, D = 304, head["D"]
    rng = np.random.default_rng(4)
    tg = rng.integers(2, head["V"], size=N).astype(np.int32)
    base = W[tg] / (W[tg] ** 2).sum(1, keepdims=True) * np.linspace(1, 40, N)[:, None]
    H = torch.from_numpy(base + 0.3 * rng.normal(size=(N, D))).to(torch.bfloat16)
    Y = oracle.logits(head, bf16_bits(H))
    m = Y.max(1)
    lse = m + np.log(np.exp(Y - m[:, None]).sum(1))
    P = np.exp(Y - lse[:, None])
    rest = P.copy()
    rest[np.arange(N), tg] = 0
    P[np.arange(N), tg] = -rest.sum(1)
    Hd, t = H.cuda(), torch.from_numpy(tg).cuda()
    parts = [ah.nll_lse(Hd[n:n + 8], dh, t[n:n + 8]) for n in range(0, N, 8)]
    nl, ls = (torch.cat(x) for x in zip(*parts))
    got = ah.nll_grad(Hd, dh, t, nl, ls, torch.ones(N, device="cuda"))
    ah.check()
    want = P @ W
    # as for confident tokens of one batch; every probability besides moves by what the two kernels'
    # logits differ by, at most 1e-4 max|Y| each
    slip = 4 * 2.0 ** -24 * np.abs(Y).max(1)[:, None]
    tol = nll_tol(head, P, Y, M, np.ones(N, np.float32), want) + 2 * slip * M[tg] + 1e-4 * np.abs(Y).max() * (np.abs(P) @ M)
    close(got, want, tol)
    assert nl.min() < 1e-3
