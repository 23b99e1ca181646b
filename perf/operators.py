"""The training operators of the packed head, as cases to measure: the gradient of the
per-token NLL and of the logits with respect to the hidden states, through the packed head,
and the losses on per-token NLLs (clipped policy loss with a KL term, paired preference
loss), each with its gradient.

`run` computes a case in its plain form, elementary torch operations on the dense head
decoded from its packed bytes, or, where `own` is true, through the package's entry points.
"""
import math

import numpy as np
import torch

own = False

POLICY = {"clip_low": 0.2, "clip_high": 0.28, "kl_coef": 0.05}


def listed():
    return [
        # one small head, one decode-sized batch: the smallest call, where latency counts
        {"name": "nll_grad tiny", "op": "nll_grad", "N": 16, "V": 4096, "D": 512, "r_c": 16, "r_r": 16, "g": 64},
        # a few scored tokens of a large head: the head's bytes bound it
        {"name": "nll_grad N64", "op": "nll_grad", "N": 64, "V": 151936, "D": 4096, "r_c": 32, "r_r": 32, "g": 128},
        # a ragged batch of sequences packed without padding, larger ranks
        {"name": "nll_grad N777", "op": "nll_grad", "N": 777, "V": 128256, "D": 4096, "r_c": 64, "r_r": 64, "g": 128},
        # one training micro-batch of 4096 tokens
        {"name": "nll_grad N4096", "op": "nll_grad", "N": 4096, "V": 151936, "D": 4096, "r_c": 32, "r_r": 32, "g": 128},
        # the wide head with a large batch: the largest call
        {"name": "nll_grad wide N8192", "op": "nll_grad", "N": 8192, "V": 151936, "D": 5120, "r_c": 32, "r_r": 32, "g": 128},
        # a user's own loss on the logits of one token
        {"name": "logits_grad N1", "op": "logits_grad", "N": 1, "V": 151936, "D": 4096, "r_c": 32, "r_r": 32, "g": 128},
        # odd vocabulary, odd batch, fine groups, ranks that are no multiple of four
        {"name": "logits_grad odd", "op": "logits_grad", "N": 331, "V": 32003, "D": 1920, "r_c": 7, "r_r": 18, "g": 32},
        # a user's own loss on the logits of a batch
        {"name": "logits_grad N1024", "op": "logits_grad", "N": 1024, "V": 128256, "D": 4096, "r_c": 64, "r_r": 64, "g": 128},
        # a few short answers
        {"name": "policy small", "op": "policy", "B": 7, "mean": 40, "ref": True, "mask": True, "per_seq": True, "reduction": "token"},
        # a large rollout batch, every sequence counting alike
        {"name": "policy large", "op": "policy", "B": 8192, "mean": 512, "ref": True, "mask": True, "per_seq": False, "reduction": "sequence"},
        # a small batch of preference pairs
        {"name": "preference small", "op": "preference", "B": 16, "mean": 60, "pairs": 8, "ref": True, "mask": True, "kind": "sigmoid", "average": False},
        # many answers to the same prompts, each compared with several others
        {"name": "preference large", "op": "preference", "B": 8192, "mean": 512, "pairs": 12000, "ref": True, "mask": True, "kind": "sigmoid", "average": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["nll_grad", "nll_grad", "logits_grad", "logits_grad", "policy", "preference"])
    if op in ("nll_grad", "logits_grad"):
        g = rng.choice([32, 64, 128, 128, 256])
        unit = max(128, g)
        return {"op": op, "N": _log(rng, 1, 4096 if op == "nll_grad" else 1024), "V": _log(rng, 1000, 151936),
                "D": unit * _log(rng, 1, 5120 // unit), "r_c": rng.choice([0, 5, 16, 32, 64, 128]),
                "r_r": rng.choice([0, 3, 16, 32, 64, 128]), "g": g}
    B = _log(rng, 2, 8192)
    case = {"op": op, "B": B, "mean": _log(rng, 1, min(4096, (1 << 22) // B)), "ref": rng.random() < 0.7,
            "mask": rng.random() < 0.7}
    if op == "policy":
        return {**case, "per_seq": rng.random() < 0.5, "reduction": rng.choice(["token", "sequence", "sum"])}
    return {**case, "pairs": _log(rng, 1, 12000), "kind": rng.choice(["sigmoid", "sigmoid", "hinge", "ipo"]),
            "average": rng.random() < 0.4}


def _generator(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def _head(case, gen):
    """A packed head in its canonical layout: normal residuals and low-rank factors that give
    logits of a few units, as language-model heads do."""
    V, D, g, G = case["V"], case["D"], case["g"], case["D"] // case["g"]
    noise = 1.28 / math.sqrt(D)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    nib = torch.empty(V, D // 2, dtype=torch.uint8, device="cuda")
    for v0 in range(0, V, 16384):
        q = (normal(min(V, v0 + 16384) - v0, D) * 2.6).round_().clamp_(-8, 7).to(torch.int8) & 15
        nib[v0:v0 + 16384] = (q[:, 0::2] | (q[:, 1::2] << 4)).view(torch.uint8)
    code = torch.randint(120, 256, (V, G), generator=gen, device="cuda", dtype=torch.uint8)
    code[:, 0] = 255
    sup = (noise / (2.6 * 190) * torch.exp(0.2 * normal(V))).to(torch.bfloat16)
    head = {"V": V, "D": D, "r_c": case["r_c"], "r_r": case["r_r"], "g": g, "r_nib": nib, "r_code": code, "r_super": sup}
    for a, b, r, share in (("Ac", "Bc", case["r_c"], 0.5), ("Aw", "Bw", case["r_r"], 0.25)):
        head[a] = (normal(V, r) * 40).round_().clamp_(-127, 127).to(torch.int8)
        head[b] = (normal(r, D) * 40).round_().clamp_(-127, 127).to(torch.int8)
        head["s" + b] = torch.exp(0.2 * normal(r, G)) / 512
        head["s" + a] = share * noise * 512 / (1600 * math.sqrt(max(r, 1))) * torch.exp(0.2 * normal(V))
    return head


def _dense(head):
    """The dense head (V x D, FP32) from the packed bytes."""
    V, D, g = head["V"], head["D"], head["g"]
    W = torch.empty(V, D, device="cuda")
    W[:, 0::2] = ((head["r_nib"] & 15).to(torch.int8) ^ 8) - 8
    W[:, 1::2] = ((head["r_nib"] >> 4).to(torch.int8) ^ 8) - 8
    W.view(V, D // g, g).mul_((head["r_code"].float() * head["r_super"].float()[:, None])[:, :, None])
    for a, b in (("Ac", "Bc"), ("Aw", "Bw")):
        if head[a].shape[1]:
            right = (head[b].float().view(-1, D // g, g) * head["s" + b][:, :, None]).view(-1, D)
            W.addmm_(head[a].float() * head["s" + a][:, None], right)
    return W


def _hidden(case, gen):
    s = torch.exp(0.5 * torch.randn(case["D"], generator=gen, device="cuda"))
    s[torch.randint(0, case["D"], (4,), generator=gen, device="cuda")] *= 20
    return (torch.randn(case["N"], case["D"], generator=gen, device="cuda") * s).to(torch.bfloat16)


def _tokens(case, gen):
    """Ragged sequences with empty ones, their token weights and per-token log-likelihoods."""
    B, mean = case["B"], case["mean"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    N = B * mean
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[1:B] = torch.randint(0, N + 1, (B - 1,), generator=gen, device="cuda").sort()[0]
    cu[B] = N
    nll = torch.nn.functional.softplus(2 * normal(N) - 1)
    state = {"cu": cu, "nll": nll, "ref": None, "w": None}
    if case["ref"]:
        state["ref"] = (nll + 0.2 * normal(N)).abs()
    if case["mask"]:  # prompts and padding do not count, and a few sequences have nothing that counts
        state["w"] = (torch.rand(N, generator=gen, device="cuda") < 0.75).float()
        state["w"][:int(cu[B // 3])] *= (torch.arange(int(cu[B // 3]), device="cuda") >= int(cu[B // 4]))
    return state, normal


def prepare(case, seed):
    gen = _generator(seed)
    op = case["op"]
    if op in ("nll_grad", "logits_grad"):
        head = _head(case, gen)
        N, V = case["N"], case["V"]
        target = torch.randint(0, V, (N,), generator=gen, device="cuda", dtype=torch.int32)
        state = {"case": case, "target": target}
        if op == "nll_grad":  # the forward pass left each token's NLL and log-sum-exp
            H, W = _hidden(case, gen), _dense(head)
            state["H"], state["nll"], state["lse"] = H, torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
            for n0 in range(0, N, 2048):
                Y = H[n0:n0 + 2048].float() @ W.T
                lse = torch.logsumexp(Y.double() if V * N < 1 << 24 else Y, 1)
                state["lse"][n0:n0 + 2048] = lse
                state["nll"][n0:n0 + 2048] = lse - Y.gather(1, target[n0:n0 + 2048, None].long())[:, 0]
            del Y, W
            counts = torch.rand(N, generator=gen, device="cuda") < 0.9
            counts[0] = True
            state["dnll"] = torch.randn(N, generator=gen, device="cuda") * counts / N
        else:  # a softmax gradient with the weights of a mean over the batch
            dY = torch.randn(N, V, generator=gen, device="cuda").mul_(2.5).exp_()
            dY.div_(dY.sum(1, keepdim=True))
            dY[torch.arange(N, device="cuda"), target.long()] -= 1
            state["dY"] = dY.mul_(torch.randn(N, 1, generator=gen, device="cuda") / N)
        if own:
            import packed_int4_lm_b200 as ah
            host = {k: v.view(torch.int16) if v.dtype == torch.bfloat16 else v for k, v in head.items() if torch.is_tensor(v)}
            host = {k: v.cpu().numpy() for k, v in host.items()}
            host["r_super"] = host["r_super"].view(np.uint16)
            state["head"] = ah.DeviceHead.from_canonical({**{k: v for k, v in head.items() if not torch.is_tensor(v)}, **host}, "cuda")
        else:
            state["head"] = head
        return state
    state, normal = _tokens(case, gen)
    state["case"] = case
    if op == "policy":
        state["old"] = (state["nll"] + 0.15 * normal(state["nll"].numel())).abs()
        state["adv"] = normal(case["B"] if case["per_seq"] else state["nll"].numel())
    else:
        state["pairs"] = torch.randint(0, case["B"], (case["pairs"], 2), generator=gen, device="cuda", dtype=torch.int32)
    return state


def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return {"nll_grad": _nll_grad, "logits_grad": _logits_grad, "policy": _policy, "preference": _preference}[op](state)


def _own(s, op):
    import packed_int4_lm_b200 as ah
    c = s["case"]
    if op == "nll_grad":
        return ah.nll_grad(s["H"], s["head"], s["target"], s["nll"], s["lse"], s["dnll"])
    if op == "logits_grad":
        return ah.logits_grad(s["dY"], s["head"])
    if op == "policy":
        return ah.policy_loss(s["nll"], s["old"], s["adv"], nll_ref=s["ref"], weights=s["w"], cu_seqlens=s["cu"],
                              per_sequence=c["per_seq"], reduction=c["reduction"], **POLICY)
    return ah.preference_loss(s["nll"], s["cu"], s["pairs"], nll_ref=s["ref"], weights=s["w"], beta=0.1,
                              kind=c["kind"], average=c["average"], margin=0.1,
                              label_smoothing=0.05 if c["kind"] == "sigmoid" else 0.0)


def _nll_grad(s):
    W = _dense(s["head"])
    P = s["H"].float() @ W.T
    P.sub_(s["lse"][:, None]).exp_()
    rows = torch.arange(P.shape[0], device="cuda")
    # 1 - p of the target cancels in 32 bits where p is near 1: the NLL says it exactly
    P[rows, s["target"].long()] = torch.expm1(-s["nll"].double()).float()
    return ((P @ W) * s["dnll"][:, None]).to(torch.bfloat16)


def _logits_grad(s):
    return (s["dY"] @ _dense(s["head"])).to(torch.bfloat16)


def _segments(s):
    """Each token's sequence."""
    at = torch.arange(s["nll"].numel(), device="cuda", dtype=torch.int32)
    return torch.searchsorted(s["cu"][1:], at, right=True)


def _policy(s):
    c = s["case"]
    nll, seg = s["nll"], _segments(s)
    adv = s["adv"][seg] if c["per_seq"] else s["adv"]
    w = s["w"].double() if s["w"] is not None else torch.ones_like(nll, dtype=torch.float64)
    # the side of the clip border and small differences of log-probs in 64 bits
    x = s["old"].double() - nll.double()
    r = torch.exp(x)
    clipped = ((adv > 0) & (x > math.log1p(POLICY["clip_high"]))) | ((adv < 0) & (x < math.log1p(-POLICY["clip_low"])))
    edge = torch.where(adv > 0, 1 + POLICY["clip_high"], 1 - POLICY["clip_low"]).double()
    surrogate = -torch.where(clipped, edge, r) * adv
    grad = torch.where(clipped, torch.zeros_like(r), r * adv)
    kl = torch.zeros_like(r)
    if s["ref"] is not None:
        z = nll.double() - s["ref"].double()
        kl = torch.expm1(z) - z
        grad = grad + POLICY["kl_coef"] * torch.expm1(z)
    if c["reduction"] == "sequence":
        total = torch.zeros(c["B"], dtype=torch.float64, device="cuda").index_add_(0, seg, w)
        scale = torch.where(total > 0, 1 / total, 0)[seg] / (total > 0).sum().clamp(min=1)
    elif c["reduction"] == "token":
        total = w.sum()
        scale = torch.where(total > 0, 1 / total, 0)
    else:
        scale = 1.0
    w = w * scale
    parts = torch.stack([(w * surrogate).sum(), (w * kl).sum(), (w * clipped).sum()])
    stats = torch.stack([parts[0] + POLICY["kl_coef"] * parts[1], parts[0], parts[1], parts[2]])
    return {"stats": stats.float(), "dnll": (w * grad).float()}


def _preference(s):
    c = s["case"]
    nll, seg = s["nll"].double(), _segments(s)
    w = s["w"].double() if s["w"] is not None else torch.ones_like(nll)
    ratio = (s["ref"].double() if s["ref"] is not None else 0) - nll
    sums = torch.zeros(c["B"], dtype=torch.float64, device="cuda")
    score, count = sums.index_add(0, seg, w * ratio), sums.index_add(0, seg, w)
    per = torch.where(count > 0, 1 / count, 0) if c["average"] else torch.ones_like(count)
    score = score * per
    a, b = s["pairs"][:, 0].long(), s["pairs"][:, 1].long()
    beta, smooth, margin = 0.1, 0.05, 0.1
    gap = score[a] - score[b]
    m = beta * gap - margin
    if c["kind"] == "sigmoid":
        loss = (1 - smooth) * torch.log1p(torch.exp(-m.abs())) + smooth * torch.log1p(torch.exp(-m.abs()))
        loss = loss + (1 - smooth) * (-m).clamp(min=0) + smooth * m.clamp(min=0)
        slope = beta * (smooth / (1 + torch.exp(-m)) - (1 - smooth) / (1 + torch.exp(m)))
    elif c["kind"] == "hinge":
        loss = (1 - m).clamp(min=0)
        slope = torch.where(m < 1, -beta, 0.0).double()
    else:
        loss = (gap - margin - 1 / (2 * beta)) ** 2
        slope = 2 * (gap - margin - 1 / (2 * beta))
    slope = slope / a.numel()
    by = sums.index_add(0, a, slope).index_add(0, b, -slope) * per
    return {"loss": loss.mean().float().view(1), "pair_loss": loss.float(),
            "rewards": (beta * torch.stack([score[a], score[b]], 1)).float(), "dnll": (-w * by[seg]).float()}


def _head_bytes(c):
    V, D, G, R = c["V"], c["D"], c["D"] // c["g"], c["r_c"] + c["r_r"]
    return V * D // 2 + V * G + 2 * V + R * (V + D) + 4 * (R * G + V * ((c["r_c"] > 0) + (c["r_r"] > 0)))


def work(case):
    op = case["op"]
    if op in ("nll_grad", "logits_grad"):
        N, V, D, R = case["N"], case["V"], case["D"], case["r_c"] + case["r_r"]
        product = 2 * N * V * D + 2 * N * R * (V + D)
        if op == "nll_grad":  # the logits again, then the gradient's product
            return {"bytes": _head_bytes(case) + 4 * N * D + 16 * N, "flops": 2 * product}
        return {"bytes": _head_bytes(case) + 4 * N * V + 2 * N * D, "flops": product}
    N = case["B"] * case["mean"]
    arrays = 2 + case["ref"] + case["mask"]  # the NLLs and their gradient
    if op == "policy":
        return {"bytes": 4 * N * (arrays + 1 + (not case["per_seq"])) + 4 * case["B"] * (1 + case["per_seq"]), "flops": 30 * N}
    return {"bytes": 4 * N * arrays + 4 * case["B"] + 20 * case["pairs"], "flops": 6 * N}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("nll_grad", "logits_grad"):
        return _exact_product(case, s)
    cu = s["cu"].cpu().numpy()
    v = {k: s[k].double().cpu().numpy() for k in ("nll", "ref", "w", "old", "adv") if s.get(k) is not None}
    N, B = len(v["nll"]), case["B"]
    w = v.get("w", np.ones(N))
    slices = [slice(cu[i], cu[i + 1]) for i in range(B)]
    if case["op"] == "policy":
        adv = np.repeat(v["adv"], np.diff(cu)) if case["per_seq"] else v["adv"]
        scale = np.ones(N)
        if case["reduction"] == "token":
            scale[:] = 1 / w.sum() if w.sum() > 0 else 0
        elif case["reduction"] == "sequence":
            totals = np.array([w[i].sum() for i in slices])
            for i, t in zip(slices, totals):
                scale[i] = 1 / t / (totals > 0).sum() if t > 0 else 0
        ratio = np.exp(v["old"] - v["nll"])
        kept = np.clip(ratio, 1 - POLICY["clip_low"], 1 + POLICY["clip_high"])
        outside = ratio * adv > kept * adv
        sur = -np.minimum(ratio * adv, kept * adv)
        grad = np.where(outside, 0, ratio * adv)
        kl = np.zeros(N)
        if "ref" in v:
            up = np.expm1(v["nll"] - v["ref"])
            kl, grad = up - (v["nll"] - v["ref"]), grad + POLICY["kl_coef"] * up
        means = [(scale * w * x).sum() for x in (sur, kl, outside)]
        return {"stats": np.array([means[0] + POLICY["kl_coef"] * means[1], *means]), "dnll": scale * w * grad}
    logratio = v.get("ref", np.zeros(N)) - v["nll"]
    count = np.array([w[i].sum() for i in slices])
    score = np.array([(w[i] * logratio[i]).sum() for i in slices])
    share = np.divide(1, count, out=np.zeros(B), where=count > 0) if case["average"] else np.ones(B)
    score, back = score * share, np.zeros(B)
    a, b = s["pairs"].cpu().numpy().T
    d = score[a] - score[b]
    m = 0.1 * d - 0.1
    if case["kind"] == "sigmoid":
        loss = 0.95 * np.logaddexp(0, -m) + 0.05 * np.logaddexp(0, m)
        slope = 0.1 * (0.05 - 1 / (1 + np.exp(m)))
    elif case["kind"] == "hinge":
        loss, slope = np.maximum(0, 1 - m), -0.1 * (m < 1)
    else:
        loss, slope = (d - 5.1) ** 2, 2 * (d - 5.1)
    np.add.at(back, a, slope / len(a))
    np.add.at(back, b, -slope / len(a))
    return {"loss": np.array([loss.mean()]), "pair_loss": loss, "rewards": 0.1 * np.stack([score[a], score[b]], 1),
            "dnll": -w * np.repeat(back * share, np.diff(cu))}


def _exact_product(case, s):
    """dH in 64 bits, a slice of the vocabulary at a time."""
    head, D, g = s["head"], case["D"], case["g"]
    right = {b: head[b].double() * head["s" + b].double().repeat_interleave(g, 1) for b in ("Bc", "Bw")}
    out = torch.zeros(case["N"], D, dtype=torch.float64, device="cuda")
    for v0 in range(0, case["V"], 8192):
        rows = slice(v0, min(case["V"], v0 + 8192))
        byte = head["r_nib"][rows].long()
        q = torch.stack([byte % 16, byte // 16], 2).flatten(1)
        q = torch.where(q > 7, q - 16, q).double()
        W = q * head["r_code"][rows].double().repeat_interleave(g, 1) * head["r_super"][rows].double()[:, None]
        for a, b in (("Ac", "Bc"), ("Aw", "Bw")):
            W += (head[a][rows].double() * head["s" + a][rows].double()[:, None]) @ right[b]
        if case["op"] == "logits_grad":
            out += s["dY"][:, rows].double() @ W
            continue
        P = torch.exp(s["H"].double() @ W.T - s["lse"].double()[:, None])
        hit = torch.nonzero((s["target"] >= rows.start) & (s["target"] < rows.stop))[:, 0]
        P[hit, s["target"][hit].long() - v0] -= 1
        out += P @ W
    return out * s["dnll"].double()[:, None] if case["op"] == "nll_grad" else out
