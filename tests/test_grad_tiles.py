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
