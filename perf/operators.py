"""What is measured of the operators on the vocabulary matrix: the log
probabilities of given tokens at the LM head (with entropy and the top
alternatives), their gradients, the scaled embedding lookup and its gradient.

``run`` computes them in plain torch operations in fp32 while ``own`` is false,
and through ``linear_cross_entropy_ce_gb300.flce`` while it is true.
"""
import math

import numpy as np
import torch

own = False

IGNORE = -100


def listed():
    return [
        # one decode step of a served sequence, with the alternatives shown to the user
        {"name": "logprobs_decode_1", "op": "logprobs", "n": 1, "h": 4096, "v": 128256, "k": 8, "ignored": 0.0,
         "temperature": 1.0},
        # one decode step of a batch over a large odd vocabulary, sampled at a temperature
        {"name": "logprobs_decode_61", "op": "logprobs", "n": 61, "h": 2048, "v": 256007, "k": 5, "ignored": 0.0,
         "temperature": 0.7},
        # scoring one sequence whose prompt is not scored, with alternatives
        {"name": "logprobs_score_1033", "op": "logprobs", "n": 1033, "h": 4096, "v": 128256, "k": 20, "ignored": 0.3,
         "temperature": 1.0},
        # scoring a batch of a small model
        {"name": "logprobs_score_4096", "op": "logprobs", "n": 4096, "h": 512, "v": 16000, "k": 0, "ignored": 0.05,
         "temperature": 1.0},
        # reference-policy log probabilities of a batch of rollouts
        {"name": "logprobs_score_16384", "op": "logprobs", "n": 16384, "h": 4096, "v": 128256, "k": 0, "ignored": 0.3,
         "temperature": 1.0},
        # policy-gradient step (log probabilities, entropies, both gradients), tiny: launch latency
        {"name": "train_300", "op": "train", "n": 300, "h": 64, "v": 512, "ignored": 0.1, "temperature": 1.0},
        # the same at a small model's head
        {"name": "train_4096_small", "op": "train", "n": 4096, "h": 512, "v": 16000, "ignored": 0.05,
         "temperature": 0.9},
        # the same at a large head
        {"name": "train_4096", "op": "train", "n": 4096, "h": 4096, "v": 128256, "ignored": 0.3, "temperature": 1.0},
        # token embedding of one decode step of a batch
        {"name": "embedding_61", "op": "embedding", "n": 61, "h": 4096, "v": 128256, "dtype": "bf16", "zipf": True},
        # token embedding of a training batch
        {"name": "embedding_65536", "op": "embedding", "n": 65536, "h": 512, "v": 16000, "dtype": "bf16",
         "zipf": True},
        # its gradient: frequent tokens take thousands of rows each
        {"name": "embedding_bwd_65536", "op": "embedding_bwd", "n": 65536, "h": 512, "v": 16000, "dtype": "bf16",
         "zipf": True},
        # its gradient at a large vocabulary: most rows are zero
        {"name": "embedding_bwd_16384", "op": "embedding_bwd", "n": 16384, "h": 4096, "v": 128256, "dtype": "bf16",
         "zipf": True},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "train", "embedding", "embedding_bwd"])
    h = 8 * _log_int(rng, 8, 512)
    v = _log_int(rng, 500, 260000)
    if op in ("logprobs", "train"):
        most = (16384 if op == "logprobs" else 4096) * 4096 * 128256
        n = min(_log_int(rng, 1, 16384 if op == "logprobs" else 4096), most // (h * v))
        c = {"op": op, "n": n, "h": h, "v": v, "ignored": rng.choice([0.0, 0.05, 0.3, 0.5]),
             "temperature": rng.choice([1.0, 0.7, 1.3])}
        if op == "logprobs":
            c["k"] = rng.randint(1, 32) if n * v <= 1 << 27 else 0
        return c
    return {"op": op, "n": _log_int(rng, 1, 65536), "h": h, "v": min(v, (128256 * 4096) // h),
            "dtype": rng.choice(["bf16", "fp16", "fp32"]), "zipf": rng.random() < 0.7}


_DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _zipf(v):
    p = np.arange(1, v + 1, dtype=np.float64) ** -1.1
    return p / p.sum()


def _ids(case, gen, dev):
    n, v = case["n"], case["v"]
    if not case.get("zipf", True):
        return torch.randint(0, v, (n,), generator=gen, device=dev, dtype=torch.int32)
    cdf = torch.cumsum(torch.arange(1, v + 1, device=dev, dtype=torch.float64) ** -1.1, 0)
    u = torch.rand(n, generator=gen, device=dev, dtype=torch.float64) * cdf[-1]
    rank = torch.searchsorted(cdf, u).clamp_(max=v - 1)
    return torch.randperm(v, generator=gen, device=dev)[rank].to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    n, h, v = case["n"], case["h"], case["v"]
    s = {"case": case}
    if case["op"] in ("logprobs", "train"):
        # Logits of standard deviation 1.28 (weights of 0.02 at a hidden size of 4096), and hidden states that
        # lean towards the row of the token that follows, some of them strongly, as those of a trained model do.
        std = 1.28 / math.sqrt(h)
        w = torch.randn((v, h), generator=gen, device=dev) * std
        t = _ids(case, gen, dev)
        lift = 14.0 * torch.rand((n, 1), generator=gen, device=dev)
        x = torch.randn((n, h), generator=gen, device=dev) + w[t.long()] * (lift / (h * std * std))
        if case.get("k", 0):
            # The ids of the top alternatives are whole numbers. Inputs on a coarse grid (as those of a quantised
            # checkpoint) make every sum of products exact in fp32 in any order, so equal logits are equal
            # everywhere and the lowest id decides.
            step = 2.0 ** round(math.log2(std / 10))
            w = torch.round(w / step).clamp_(-63, 63) * step
            x = torch.round(x * 16).clamp_(-64, 64) / 16
        s["weight"], s["hidden"] = w.to(torch.bfloat16), x.to(torch.bfloat16)
        # the first tokens of every sequence of up to 1024 tokens are the prompt, which is not scored
        seq = min(n, 1024)
        prompt = torch.arange(n, device=dev) % seq < int(case["ignored"] * seq)
        s["targets"] = torch.where(prompt, torch.full_like(t, IGNORE), t)
        if case["op"] == "train":
            s["grad_logp"] = -torch.randn(n, generator=gen, device=dev) / n          # advantages
            s["grad_entropy"] = -0.1 * torch.rand(n, generator=gen, device=dev) / n  # entropy bonus
        return s
    dt = _DTYPE[case["dtype"]]
    s["ids"] = _ids(case, gen, dev)
    s["scale"] = math.sqrt(h)
    if case["op"] == "embedding":
        s["weight"] = (torch.randn((v, h), generator=gen, device=dev) * 0.02).to(dt)
    else:
        s["grad_out"] = torch.randn((n, h), generator=gen, device=dev).to(dt)
    return s


def _run_own(s):
    from linear_cross_entropy_ce_gb300 import flce
    c = s["case"]
    if c["op"] == "logprobs":
        o = flce.token_logprobs(s["hidden"], s["weight"], s["targets"], IGNORE, temperature=c["temperature"],
                                top_k=c["k"])
        r = {"logp": o["logp"], "entropy": o["entropy"]}
        if c["k"]:
            r["top_ids"], r["top_logp"] = o["top_ids"], o["top_logp"]
        return r
    if c["op"] == "train":
        o = flce.token_logprobs(s["hidden"], s["weight"], s["targets"], IGNORE, temperature=c["temperature"])
        g = flce.token_logprobs_bwd(s["hidden"], s["weight"], s["targets"], o["lse"], o["entropy"], s["grad_logp"],
                                    s["grad_entropy"], IGNORE, temperature=c["temperature"],
                                    grad_weight_dtype=torch.bfloat16)
        return {"logp": o["logp"], "entropy": o["entropy"], "grad_hidden": g["grad_hidden"],
                "grad_weight": g["grad_weight"]}
    if c["op"] == "embedding":
        return flce.embedding_fwd(s["weight"], s["ids"], s["scale"])
    return flce.embedding_bwd(s["grad_out"], s["ids"], c["v"], s["scale"])["grad_weight"]


def _plain_logprobs(s):
    c = s["case"]
    t = s["targets"].long()
    valid = t != IGNORE
    x, w = s["hidden"].float(), s["weight"].float()
    z = (x @ w.T) / c["temperature"]
    m = z.max(dim=1, keepdim=True).values
    lse = m + torch.log(torch.exp(z - m).sum(dim=1, keepdim=True))
    lp = z - lse
    p = torch.exp(lp)
    ent = -(p * lp).sum(dim=1, keepdim=True)
    at = torch.where(valid, t, 0)[:, None]
    return valid[:, None], x, w, at, lp, p, ent


def run(s):
    if own:
        return _run_own(s)
    c = s["case"]
    if c["op"] == "logprobs":
        valid, x, w, at, lp, p, ent = _plain_logprobs(s)
        r = {"logp": torch.where(valid, lp.gather(1, at), 0.0)[:, 0], "entropy": torch.where(valid, ent, 0.0)[:, 0]}
        if c["k"]:
            top, ids = torch.sort(lp, dim=1, descending=True, stable=True)
            r["top_ids"] = torch.where(valid, ids[:, :c["k"]], -1).to(torch.int32)
            r["top_logp"] = torch.where(valid, top[:, :c["k"]], 0.0)
        return r
    if c["op"] == "train":
        valid, x, w, at, lp, p, ent = _plain_logprobs(s)
        g = torch.where(valid, s["grad_logp"][:, None], 0.0)
        e = torch.where(valid, s["grad_entropy"][:, None], 0.0)
        dz = -p * (g + e * (lp + ent))
        dz.scatter_add_(1, at, g)
        dz = dz / c["temperature"]
        return {"logp": torch.where(valid, lp.gather(1, at), 0.0)[:, 0], "entropy": torch.where(valid, ent, 0.0)[:, 0],
                "grad_hidden": (dz @ w).to(torch.bfloat16), "grad_weight": (dz.T @ x).to(torch.bfloat16)}
    if c["op"] == "embedding":
        w = s["weight"]
        return (w[s["ids"].long()].float() * s["scale"]).to(w.dtype)
    g = torch.zeros((c["v"], c["h"]), device=s["grad_out"].device)
    return g.index_add_(0, s["ids"].long(), s["grad_out"].float()) * s["scale"]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "embedding":
        return torch.nn.functional.embedding(s["ids"].long(), s["weight"].double()) * s["scale"]
    if case["op"] == "embedding_bwd":
        # by sorted ids: differences of running sums are taken within each id only
        order = torch.argsort(s["ids"], stable=True)
        rows = s["grad_out"].double()[order]
        ids, count = torch.unique_consecutive(s["ids"][order], return_counts=True)
        sums = torch.segment_reduce(rows, "sum", lengths=count, axis=0)
        g = torch.zeros((case["v"], case["h"]), device=rows.device, dtype=torch.float64)
        g[ids.long()] = sums * s["scale"]
        return g
    n, h, v = case["n"], case["h"], case["v"]
    keep = torch.nonzero(s["targets"] != IGNORE)[:, 0]
    if (2 if case["op"] == "logprobs" else 6) * keep.numel() * h * v > 1.4e13:
        return None
    x, w = s["hidden"][keep].double(), s["weight"].double()
    train = case["op"] == "train"
    with torch.set_grad_enabled(train):
        x.requires_grad_(train)
        w.requires_grad_(train)
        lp = torch.log_softmax(x @ w.T / case["temperature"], dim=1)
        logp = lp[torch.arange(keep.numel(), device=lp.device), s["targets"][keep].long()]
        ent = torch.special.entr(lp.exp()).sum(1)
        if train:
            ((logp * s["grad_logp"][keep]).sum() + (ent * s["grad_entropy"][keep]).sum()).backward()

    def rows(a, fill=0):
        full = torch.full((n,) + a.shape[1:], fill, device=a.device, dtype=a.dtype)
        full[keep] = a.detach()
        return full

    r = {"logp": rows(logp), "entropy": rows(ent)}
    if train:
        return {**r, "grad_hidden": rows(x.grad), "grad_weight": w.grad}
    if case["k"]:
        r["top_ids"] = None
        top = torch.topk(lp, case["k"], dim=1).values
        r["top_logp"] = rows(top)
    return r


def work(case):
    n, h, v = case["n"], case["h"], case["v"]
    if case["op"] in ("logprobs", "train"):
        seq = min(n, 1024)
        prompt = int(case["ignored"] * seq)
        nv = n - (n // seq) * prompt - min(n % seq, prompt)
        if case["op"] == "logprobs":
            return {"bytes": 2 * h * (nv + v) + 12 * n + 8 * n * case["k"], "flops": 2 * nv * h * v}
        return {"bytes": 2 * h * (2 * n + 2 * v) + 20 * n, "flops": 6 * nv * h * v}
    size = 4 if case["dtype"] == "fp32" else 2
    p = _zipf(v) if case["zipf"] else np.full(v, 1.0 / v)
    distinct = float(np.sum(-np.expm1(n * np.log1p(-p)))) if v > 1 else 1.0
    if case["op"] == "embedding":
        return {"bytes": size * h * (distinct + n) + 4 * n, "flops": n * h}
    return {"bytes": size * h * n + 4 * n + 4 * h * v, "flops": n * h}
