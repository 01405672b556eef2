"""What is measured of the operators on next-token distributions at the LM head:
the log probabilities and top alternatives under penalties for repeated tokens,
biases and grammar masks (serving), and the distillation loss from a teacher's
top log probabilities with its gradients (training).

``run`` computes them in plain torch operations in fp32 while ``own`` is false,
and through ``linear_cross_entropy_ce_gb300.flce`` while it is true.
"""
import math

import torch

own = False

IGNORE = -100


def listed():
    return [
        # one decode step of a short chat turn: a few dozen tokens of history, the alternatives shown to the user
        {"name": "constrained_decode_1", "op": "constrained", "n": 1, "h": 4096, "v": 128256, "k": 8, "hist": 57,
         "mask": False, "bias": 0, "temperature": 1.0, "score": False},
        # one decode step of a batch over a large odd vocabulary: half of the sequences follow a grammar
        {"name": "constrained_decode_61", "op": "constrained", "n": 61, "h": 2048, "v": 256007, "k": 5, "hist": 1500,
         "mask": True, "bias": 5, "temperature": 0.7, "score": False},
        # one decode step of a full batch with long histories, grammars and bias lists
        {"name": "constrained_decode_128", "op": "constrained", "n": 128, "h": 4096, "v": 128256, "k": 20,
         "hist": 4001, "mask": True, "bias": 16, "temperature": 1.0, "score": False},
        # one decode step of a large batch of a small model
        {"name": "constrained_decode_300", "op": "constrained", "n": 300, "h": 512, "v": 16000, "k": 32, "hist": 700,
         "mask": True, "bias": 0, "temperature": 1.3, "score": False},
        # scoring a sampled sequence under the distribution it was sampled from: every position's history is the
        # sequence before it
        {"name": "constrained_score_2048", "op": "constrained", "n": 2048, "h": 4096, "v": 128256, "k": 0,
         "hist": 900, "mask": True, "bias": 0, "temperature": 1.0, "score": True},
        # distillation loss of a short answer, for evaluation
        {"name": "distill_eval_37", "op": "distill", "n": 37, "h": 4096, "v": 128256, "k": 20, "tail": True,
         "ignored": 0.0, "temperature": 1.0},
        # the same of an evaluation batch over a large odd vocabulary
        {"name": "distill_eval_8192", "op": "distill", "n": 8192, "h": 2048, "v": 256007, "k": 32, "tail": True,
         "ignored": 0.3, "temperature": 1.0},
        # distillation step (loss, both gradients), tiny: launch latency
        {"name": "distill_train_300", "op": "distill_train", "n": 300, "h": 64, "v": 512, "k": 8, "tail": False,
         "ignored": 0.1, "temperature": 2.0},
        # one odd sequence over a large odd vocabulary, many alternatives
        {"name": "distill_train_1033", "op": "distill_train", "n": 1033, "h": 2048, "v": 256007, "k": 100,
         "tail": True, "ignored": 0.3, "temperature": 1.0},
        # a batch of a small model
        {"name": "distill_train_4096_small", "op": "distill_train", "n": 4096, "h": 512, "v": 16000, "k": 20,
         "tail": False, "ignored": 0.05, "temperature": 1.5},
        # a batch at a large head
        {"name": "distill_train_4096", "op": "distill_train", "n": 4096, "h": 4096, "v": 128256, "k": 64,
         "tail": True, "ignored": 0.3, "temperature": 1.0},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["constrained", "distill", "distill_train"])
    h = 8 * _log_int(rng, 8, 512)
    v = _log_int(rng, 500, 260000)
    if op == "constrained":
        n = max(1, min(_log_int(rng, 1, 2048), (2048 * 4096 * 128256) // (h * v)))
        score = n > 1 and rng.random() < 0.25
        return {"op": op, "n": n, "h": h, "v": v, "k": 0 if score and n * v > 1 << 27 else rng.randint(0, 32),
                "hist": min(_log_int(rng, 1, 8192), (1 << 21) // n), "mask": rng.random() < 0.6,
                "bias": rng.choice([0, 0, 3, 40]), "temperature": rng.choice([1.0, 0.7, 1.3]), "score": score}
    most = (8192 * 2048 * 256007) if op == "distill" else (4096 * 4096 * 128256)
    n = max(1, min(_log_int(rng, 1, 8192), most // (h * v)))
    return {"op": op, "n": n, "h": h, "v": v, "k": _log_int(rng, 1, 200), "tail": rng.random() < 0.6,
            "ignored": rng.choice([0.0, 0.05, 0.3]), "temperature": rng.choice([1.0, 1.5, 2.0])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _zipf_ids(v, shape, gen, dev):
    cdf = torch.cumsum(torch.arange(1, v + 1, device=dev, dtype=torch.float64) ** -1.1, 0)
    u = torch.rand(shape, generator=gen, device=dev, dtype=torch.float64) * cdf[-1]
    rank = torch.searchsorted(cdf, u).clamp_(max=v - 1)
    return torch.randperm(v, generator=gen, device=dev)[rank].to(torch.int32)


def _head(n, h, v, tokens, gen, dev, grid):
    """Weights of logits of standard deviation 1.28 and hidden states that lean towards the given tokens, some of
    them strongly, as those of a trained model do.  On a coarse grid (as those of a quantised checkpoint) every sum
    of products is exact in fp32 in any order, so that equal logits are equal everywhere."""
    std = 1.28 / math.sqrt(h)
    w = torch.randn((v, h), generator=gen, device=dev) * std
    lift = 14.0 * torch.rand((n, 1), generator=gen, device=dev)
    x = torch.randn((n, h), generator=gen, device=dev) + w[tokens.long()] * (lift / (h * std * std))
    if grid:
        step = 2.0 ** round(math.log2(std / 10))
        w = torch.round(w / step).clamp_(-63, 63) * step
        x = torch.round(x * 16).clamp_(-64, 64) / 16
    return x.to(torch.bfloat16), w.to(torch.bfloat16)


def _pack(allowed):
    """[n, v] truth values as int32 words, token 0 in the lowest bit of the first."""
    n, v = allowed.shape
    words = (v + 31) // 32
    out = torch.empty((n, words), dtype=torch.int32, device=allowed.device)
    weights = torch.ones(32, dtype=torch.int64, device=allowed.device) << torch.arange(32, device=allowed.device)
    for i in range(0, n, 128):
        bits = torch.nn.functional.pad(allowed[i:i + 128], (0, words * 32 - v)).view(-1, words, 32)
        w = (bits * weights).sum(2)
        out[i:i + 128] = torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)
    return out


def _constrained_inputs(case, gen, dev):
    n, h, v = case["n"], case["h"], case["v"]
    follows = _zipf_ids(v, (n,), gen, dev)
    s = {"case": case}
    s["hidden"], s["weight"] = _head(n, h, v, follows, gen, dev, grid=True)
    if case["score"]:
        # one sequence of a prompt and the n scored tokens; position i has seen the prompt and i of them
        prompt = torch.cat([_zipf_ids(v, (case["hist"],), gen, dev), follows])
        s["history"] = prompt[None, :].expand(n, -1)
        s["history_lens"] = case["hist"] + torch.arange(n, device=dev, dtype=torch.int32)
        s["prompt_lens"] = torch.full((n,), case["hist"], device=dev, dtype=torch.int32)
        s["targets"] = follows
    else:
        s["history"] = _zipf_ids(v, (n, case["hist"]), gen, dev)
        s["history_lens"] = (case["hist"] * torch.rand(n, generator=gen, device=dev) ** 0.5 + 0.5).to(torch.int32)
        s["prompt_lens"] = (s["history_lens"] * torch.rand(n, generator=gen, device=dev)).to(torch.int32)
        s["targets"] = None
    s["repetition_penalty"] = 1.0 + 0.3 * torch.rand(n, generator=gen, device=dev)
    s["frequency_penalty"] = 0.5 * torch.rand(n, generator=gen, device=dev)
    s["presence_penalty"] = 0.6 * torch.rand(n, generator=gen, device=dev)
    s["bias_ids"] = s["bias"] = s["mask"] = None
    if case["bias"]:
        # different tokens, more or less likely, one in eight banned
        start = torch.randint(0, v, (n, 1), generator=gen, device=dev)
        s["bias_ids"] = ((start + max(1, v // 64) * torch.arange(case["bias"], device=dev)) % v).to(torch.int32)
        s["bias"] = 4.0 * torch.randn((n, case["bias"]), generator=gen, device=dev)
        if not case["score"]:
            s["bias"][torch.rand(s["bias"].shape, generator=gen, device=dev) < 0.125] = -math.inf
    if case["mask"]:
        # sequences without a grammar, inside a free string, and where few tokens may follow
        share = torch.tensor([1.0, 0.9, 0.02], device=dev)[torch.randint(0, 3, (n,), generator=gen, device=dev)]
        words = []
        for i in range(0, n, 128):
            sh = share[i:i + 128, None]
            u = torch.rand((sh.shape[0], v), generator=gen, device=dev)
            allowed = u < sh
            allowed |= torch.arange(v, device=dev) % max(1, v // 200) == 0   # more than the alternatives asked for
            if case["score"]:
                allowed[torch.arange(sh.shape[0], device=dev), follows[i:i + 128].long()] = True
            words.append(_pack(allowed))
        s["mask"] = torch.cat(words)
    return s


def _distill_inputs(case, gen, dev):
    n, h, v, k = case["n"], case["h"], case["v"], case["k"]
    k = min(k, v)
    s = {"case": case}
    x, w = _head(n, h, v, _zipf_ids(v, (n,), gen, dev), gen, dev, grid=False)
    # The teacher sees what the student sees and more: a student that has its training before it.
    t = x.float() + 1.5 * torch.randn((n, h), generator=gen, device=dev)
    ids = torch.empty((n, k), dtype=torch.int32, device=dev)
    logp = torch.empty((n, k), device=dev)
    for i in range(0, n, 512):
        z = (t[i:i + 512].to(torch.bfloat16) @ w.T).float() / case["temperature"]
        top = torch.topk(z, k, dim=1)
        ids[i:i + 512] = top.indices.to(torch.int32)
        logp[i:i + 512] = top.values - torch.logsumexp(z, 1, keepdim=True)
    # the first tokens of every sequence of up to 1024 tokens are the prompt, for which there is no teacher
    seq = min(n, 1024)
    prompt = torch.arange(n, device=dev) % seq < int(case["ignored"] * seq)
    ids[prompt] = -1
    logp[prompt] = 0.0
    s["hidden"], s["weight"], s["teacher_ids"], s["teacher_logp"] = x, w, ids, logp
    s["grad_kl"] = torch.rand(n, generator=gen, device=dev) * 2 / n   # the tokens' weights
    return s


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    return (_constrained_inputs if case["op"] == "constrained" else _distill_inputs)(case, gen, dev)


# ---------------------------------------------------------------------------
# the calls of a user
# ---------------------------------------------------------------------------

def _run_own(s):
    from linear_cross_entropy_ce_gb300 import flce
    c = s["case"]
    if c["op"] == "constrained":
        o = flce.constrained_logprobs(
            s["hidden"], s["weight"], s["targets"], IGNORE, history=s["history"], history_lens=s["history_lens"],
            prompt_lens=s["prompt_lens"], repetition_penalty=s["repetition_penalty"],
            frequency_penalty=s["frequency_penalty"], presence_penalty=s["presence_penalty"], bias_ids=s["bias_ids"],
            bias=s["bias"], mask=s["mask"], temperature=c["temperature"], top_k=c["k"])
        r = {"lse": o["lse"], "entropy": o["entropy"]}
        if s["targets"] is not None:
            r["logp"] = o["logp"]
        if c["k"]:
            r["top_ids"], r["top_logp"] = o["top_ids"], o["top_logp"]
        return r
    f = flce.topk_distill(s["hidden"], s["weight"], s["teacher_ids"], s["teacher_logp"], temperature=c["temperature"],
                          tail=c["tail"])
    r = {"kl": f["kl"], "student_logp": f["student_logp"]}
    if c["op"] == "distill_train":
        g = flce.topk_distill_bwd(s["hidden"], s["weight"], s["teacher_ids"], s["teacher_logp"], f["lse"],
                                  f["rest_logp"], f["student_logp"], s["grad_kl"], temperature=c["temperature"],
                                  tail=c["tail"], grad_weight_dtype=torch.bfloat16)
        r["grad_hidden"], r["grad_weight"] = g["grad_hidden"], g["grad_weight"]
    return r


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _logsumexp(z):
    m = z.max(dim=1, keepdim=True).values
    return m + torch.log(torch.exp(z - m).sum(dim=1, keepdim=True))


def _logsumexp64(z):
    m = z.max(dim=1, keepdim=True).values
    return m.double() + torch.log(torch.exp(z - m).sum(dim=1, keepdim=True).double())


def _plain_constrained(s):
    c = s["case"]
    n, v = c["n"], c["v"]
    z = s["hidden"].float() @ s["weight"].float().T
    at = torch.arange(s["history"].shape[1], device=z.device)[None, :]
    seen = (at < s["history_lens"][:, None]).float()
    out = seen * (at >= s["prompt_lens"][:, None])
    ids = s["history"].long()
    seen = torch.zeros_like(z).scatter_add_(1, ids, seen) > 0
    count = torch.zeros_like(z).scatter_add_(1, ids, out)
    r = s["repetition_penalty"][:, None]
    z = torch.where(seen, torch.where(z > 0, z / r, z * r), z)
    z = z - s["frequency_penalty"][:, None] * count
    z = z - s["presence_penalty"][:, None] * (count > 0)
    del seen, count
    if s["bias"] is not None:
        z = z.scatter_add_(1, s["bias_ids"].long(), s["bias"])
    if s["mask"] is not None:
        bits = (s["mask"][:, :, None] >> torch.arange(32, device=z.device, dtype=torch.int32)) & 1
        z = torch.where(bits.view(n, -1)[:, :v] != 0, z, -math.inf)
        del bits
    r = {}
    if c["k"]:
        top, ids = torch.sort(z, dim=1, descending=True, stable=True)
        r["top_ids"] = ids[:, :c["k"]].to(torch.int32)
        r["top_logp"] = top[:, :c["k"]].clone() / c["temperature"]
        del top, ids
    z = z / c["temperature"]
    lse = _logsumexp(z)
    lp = z - lse
    r["lse"] = lse[:, 0]
    r["entropy"] = -torch.where(lp > -math.inf, torch.exp(lp) * lp, 0.0).sum(1)
    if c["k"]:
        r["top_logp"] = r["top_logp"] - lse
    if s["targets"] is not None:
        r["logp"] = lp.gather(1, s["targets"].long()[:, None])[:, 0]
    return r


def _plain_distill(s):
    c = s["case"]
    ids = s["teacher_ids"].long()
    there = ids >= 0
    at = torch.where(there, ids, 0)
    valid = there.any(1)
    x, w = s["hidden"].float(), s["weight"].float()
    z = (x @ w.T) / c["temperature"]
    listed_ = torch.zeros_like(z).scatter_add_(1, at, there.float()) > 0
    # A row's own numbers in 64 bits: the divergence of two distributions that nearly agree is what is left of terms
    # far larger than itself, and the mass behind the list what is left of 1.
    lse = _logsumexp64(z)
    student = torch.where(there, z.gather(1, at) - lse, 0.0)
    t = torch.where(there, s["teacher_logp"].double(), -math.inf)
    if c["tail"]:
        p = torch.exp(t)
        r = torch.where(valid[:, None], (1.0 - p.sum(1, keepdim=True)).clamp(min=0.0), 0.0)
        rest = _logsumexp64(torch.where(listed_, -math.inf, z)) - lse
    else:
        e = torch.exp(t - torch.where(valid[:, None], t.max(dim=1, keepdim=True).values, 0.0))
        p = e / torch.where(valid[:, None], e.sum(1, keepdim=True), 1.0)
        r, rest = torch.zeros_like(lse), torch.zeros_like(lse)
    kl = torch.where(p > 0, p * (torch.log(p) - student), 0.0).sum(1)
    kl = kl + torch.where(r > 0, r * (torch.log(r) - rest), 0.0)[:, 0]
    out = {"kl": torch.where(valid, kl, 0.0).float(), "student_logp": student.float()}
    if c["op"] == "distill_train":
        g = torch.where(valid, s["grad_kl"], 0.0)[:, None] / c["temperature"]
        mass = p.sum(1, keepdim=True) + r
        dz = torch.exp(z - lse.float())
        others = (mass - r * torch.exp(-rest)).float()   # of a token behind the list
        dz = dz * torch.where(listed_, mass.float(), others)
        dz = dz.scatter_add_(1, at, -p.float()) * g
        out["grad_hidden"], out["grad_weight"] = (dz @ w).to(torch.bfloat16), (dz.T @ x).to(torch.bfloat16)
    return out


def run(s):
    if own:
        return _run_own(s)
    return _plain_constrained(s) if s["case"]["op"] == "constrained" else _plain_distill(s)


# ---------------------------------------------------------------------------
# in 64 bits, from the definitions
# ---------------------------------------------------------------------------

def _exact_constrained(s):
    c = s["case"]
    n, v, k = c["n"], c["v"], c["k"]
    if 2 * n * c["h"] * v > 1.4e13:
        return None
    z = s["hidden"].double() @ s["weight"].double().T
    lens, first = s["history_lens"].tolist(), s["prompt_lens"].tolist()
    rep, freq, pres = (s[x + "_penalty"].double() for x in ("repetition", "frequency", "presence"))
    for i in range(n):
        said = s["history"][i, :lens[i]].long()
        if said.numel():
            u = torch.unique(said)
            z[i, u] = torch.where(z[i, u] > 0, z[i, u] / rep[i], z[i, u] * rep[i])
        if lens[i] > first[i]:
            u, times = torch.unique(said[first[i]:], return_counts=True)
            z[i, u] -= freq[i] * times + pres[i]
    if s["bias"] is not None:
        rows = torch.arange(n, device=z.device)[:, None]
        z[rows, s["bias_ids"].long()] += s["bias"].double()
    if s["mask"] is not None:
        tokens = torch.arange(v, device=z.device)
        for i in range(n):
            word = s["mask"][i].long()[tokens // 32]
            z[i].masked_fill_(((word >> (tokens % 32)) & 1) == 0, -math.inf)
    z /= c["temperature"]
    lse = torch.logsumexp(z, 1)
    r = {}
    if k:
        r["top_ids"] = None
        r["top_logp"] = torch.topk(z, k, dim=1).values - lse[:, None]
    r["lse"] = lse
    r["entropy"] = torch.cat([torch.special.entr(torch.softmax(b, 1)).sum(1) for b in z.split(256)])
    if s["targets"] is not None:
        r["logp"] = z[torch.arange(n, device=z.device), s["targets"].long()] - lse
    return r


def _exact_distill(s):
    c = s["case"]
    n, h, v = c["n"], c["h"], c["v"]
    train = c["op"] == "distill_train"
    keep = torch.nonzero(s["teacher_ids"][:, 0] >= 0)[:, 0]
    if (6 if train else 2) * keep.numel() * h * v > 1.4e13:
        return None
    ids, t = s["teacher_ids"][keep].long(), s["teacher_logp"][keep].double()
    p = torch.exp(t) if c["tail"] else torch.softmax(t, 1)
    x, w = s["hidden"][keep].double(), s["weight"].double()
    with torch.set_grad_enabled(train):
        x.requires_grad_(train)
        w.requires_grad_(train)
        z = x @ w.T / c["temperature"]
        lse = torch.logsumexp(z, 1, keepdim=True)
        student = z.gather(1, ids) - lse
        kl = (torch.special.xlogy(p, p) - p * student).sum(1)
        if c["tail"]:
            r = (1 - p.sum(1)).clamp(min=0)
            others = torch.logsumexp(z.scatter(1, ids, -math.inf), 1) - lse[:, 0]
            kl = kl + torch.where(r > 0, torch.special.xlogy(r, r) - r * others, 0.0)
        if train:
            (kl * s["grad_kl"][keep].double()).sum().backward()

    def rows(a):
        full = torch.zeros((n,) + a.shape[1:], device=a.device, dtype=a.dtype)
        full[keep] = a.detach()
        return full

    out = {"kl": rows(kl), "student_logp": rows(student)}
    if train:
        out["grad_hidden"], out["grad_weight"] = rows(x.grad), w.grad
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_constrained(s) if case["op"] == "constrained" else _exact_distill(s)


def work(case):
    n, h, v, k = case["n"], case["h"], case["v"], case["k"]
    if case["op"] == "constrained":
        seen = n + case["hist"] if case["score"] else n * case["hist"] * 2 // 3
        return {"bytes": 2 * h * (n + v) + 4 * seen + (n * v // 8 if case["mask"] else 0) + 8 * n * case["bias"] +
                8 * n * (k + 4), "flops": 2 * n * h * v}
    seq = min(n, 1024)
    prompt = int(case["ignored"] * seq)
    nv = n - (n // seq) * prompt - min(n % seq, prompt)
    lists = 12 * n * min(k, v)
    if case["op"] == "distill":
        return {"bytes": 2 * h * (nv + v) + lists + 4 * n, "flops": 2 * nv * h * v}
    return {"bytes": 2 * h * (2 * n + 2 * v) + lists + 8 * n, "flops": 6 * nv * h * v}
