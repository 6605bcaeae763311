"""Cases for the operators that train the draft head, with their plain forms.

Three operators make up a training step of the head beside its objective:

linear_ce   softmax cross entropy of z = X W (+ U) over a vocabulary of V, with
            the gradients of X and W; the logits are not kept. X [N, K] holds a
            row per training position: the Markov rows W1[x_{k-1}] alone (K = r,
            U the frozen parallel logits), the hidden state alone (K = H), or
            the two side by side (K = H + r).
embed       rows of a table looked up by token and scaled, and the gradient of
            the table: the rows of the output's gradient summed per token.
clip        the 2-norm over all gradients together, and the gradients scaled to
            a largest norm.

`own` false: elementary torch operations in 32 bits. `own` true: the calls of
speculative_decoding_head_gb300.binding.
"""

import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": BF16, "f32": F32}
LARGEST_CE = 4096 * 5376 * 129280     # N K V of the largest cross entropy
LARGEST_EMBED = 262144 * 256          # N D of the largest embedding gradient
LARGEST_CLIP = 1 << 29                # values of the largest clip


def listed():
    return [
        # the head's smallest round (B = 2, gamma = 3, hidden 64, rank 16, V = 1024): latency
        {"name": "ce_step_tiny", "op": "ce", "N": 6, "K": 80, "V": 1024, "layout": "vk", "U": False, "grad": "xw",
         "ignored": 0.0, "weighted": True},
        # evaluation of the loss alone on a small batch (32 x 5 positions, hidden 1024)
        {"name": "ce_eval_small", "op": "ce", "N": 160, "K": 1024, "V": 32000, "layout": "vk", "U": False, "grad": "",
         "ignored": 0.0, "weighted": False},
        # the Markov head on frozen parallel logits: X = W1[x_prev], W = W2 as the draft reads it ([r, V])
        {"name": "ce_step_markov", "op": "ce", "N": 640, "K": 256, "V": 129280, "layout": "kv", "U": True, "grad": "xw",
         "ignored": 0.0, "weighted": True},
        # hidden state against a frozen output matrix, ragged in every size, padded rows among the tokens
        {"name": "ce_dx_ragged", "op": "ce", "N": 1001, "K": 4100, "V": 50257, "layout": "vk", "U": False, "grad": "x",
         "ignored": 0.2, "weighted": False},
        # a long training batch through hidden state and Markov row together (K = 5120 + 256)
        {"name": "ce_step_long", "op": "ce", "N": 4096, "K": 5376, "V": 129280, "layout": "vk", "U": False, "grad": "xw",
         "ignored": 0.05, "weighted": True},
        # W1 rows of a training batch (128 x 15 positions)
        {"name": "embed_rows", "op": "embed", "N": 1920, "D": 256, "V": 151936, "type": "bf16", "ld": 256, "pad": 0.0},
        # a wide embedding table, scaled, written beside other columns of the same rows
        {"name": "embed_wide", "op": "embed", "N": 16384, "D": 5120, "V": 129280, "type": "bf16", "ld": 5376, "pad": 0.02},
        # the gradient of W1 at the smallest round, all fp32
        {"name": "embed_grad_tiny", "op": "embed_grad", "N": 6, "D": 16, "V": 1024, "type": "f32", "out": "f32", "ld": 80,
         "add": False, "pad": 0.0},
        # the gradient of W1 over a long batch; frequent tokens hold a large share of the rows
        {"name": "embed_grad_long", "op": "embed_grad", "N": 262144, "D": 256, "V": 129280, "type": "bf16", "out": "bf16",
         "ld": 256, "add": False, "pad": 0.1},
        # added to a gradient that is there already, odd width, fp32 sums kept
        {"name": "embed_grad_add", "op": "embed_grad", "N": 8190, "D": 1001, "V": 32000, "type": "bf16", "out": "f32",
         "ld": 1001, "add": True, "pad": 0.0},
        # the head's own gradients (W1, W2, w, and the RNN head's Wr) at rank 256, hidden 5120, V = 129280
        {"name": "clip_head", "op": "clip", "count": 4, "total": 2 * 129280 * 256 + 5376 + 3 * 256 * 5632, "type": "bf16",
         "max_norm": 1.0, "spread": "head"},
        # many tensors of uneven sizes and both types
        {"name": "clip_many", "op": "clip", "count": 301, "total": 400000003, "type": "mixed", "max_norm": 0.5,
         "spread": "uneven"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ce", "ce", "embed", "embed_grad", "clip"])
    if op == "ce":
        while True:
            N, K, V = _log(rng, 1, 8192), _log(rng, 16, 6144), _log(rng, 256, 152000)
            if N * K * V <= LARGEST_CE:
                break
        return {"op": op, "N": N, "K": K, "V": V, "layout": rng.choice(["vk", "kv"]), "U": rng.random() < 0.3,
                "grad": rng.choice(["xw", "xw", "x", "w", ""]), "ignored": rng.choice([0.0, 0.0, 0.1, 0.5]),
                "weighted": rng.random() < 0.5}
    if op in ("embed", "embed_grad"):
        while True:
            N, D, V = _log(rng, 1, 262144), _log(rng, 8, 5120), _log(rng, 256, 152000)
            if N * D <= LARGEST_EMBED and V * D <= LARGEST_EMBED * (2 if op == "embed_grad" else 8):
                break
        c = {"op": op, "N": N, "D": D, "V": V, "type": rng.choice(["bf16", "bf16", "f32"]),
             "ld": D + rng.choice([0, 0, 8, 5]), "pad": rng.choice([0.0, 0.1])}
        if op == "embed_grad":
            c["out"] = rng.choice([c["type"], "f32"])
            c["add"] = rng.random() < 0.3
        return c
    return {"op": op, "count": _log(rng, 1, 400), "total": _log(rng, 4096, LARGEST_CLIP), "type": rng.choice(["bf16", "f32", "mixed"]),
            "max_norm": rng.choice([0.5, 1.0, 1e4]), "spread": "uneven"}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, std, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _tokens(g, n, V, pad):
    """Token ids with frequencies that fall as 1 / rank; a share `pad` of the rows holds none (-1)."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    t = (torch.exp(u * math.log(V + 1)) - 1).long().clamp_(0, V - 1)
    t = (t * 7919 + 12345) % V if V % 7919 else t
    if pad:
        t = torch.where(torch.rand(n, generator=g, device="cuda") < pad, torch.full_like(t, -1), t)
    return t.int()


def _up(x, m):
    return (x + m - 1) // m * m


def _sizes(case):
    n, total = case["count"], case["total"]
    if case["spread"] == "head":
        w = 5376
        wr = 3 * 256 * 5632
        return [(total - w - wr) // 2, (total - w - wr) // 2, w, wr]
    # sizes fall off geometrically over a factor of about 1000, each a value of its own
    f = [math.exp(-6.9 * i / n) for i in range(n)]
    s = [max(1, int(total * x / sum(f))) for x in f]
    s[0] += max(0, total - sum(s))
    return s


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "ce":
        N, K, V = case["N"], case["K"], case["V"]
        kp, vp = _up(K, 8), _up(V, 8)
        s["X"] = _normal(g, (N, kp), 1.0, BF16)[:, :K]
        s["W"] = (_normal(g, (V, kp), 2.0 / math.sqrt(K), BF16)[:, :K] if case["layout"] == "vk"
                  else _normal(g, (K, vp), 2.0 / math.sqrt(K), BF16)[:, :V])
        s["U"] = _normal(g, (N, _up(V, 4)), 2.0, F32)[:, :V] if case["U"] else None
        s["target"] = _tokens(g, N, V, case["ignored"])
        # position k of a block weighs exp(-k / 4), blocks of five positions
        s["wt"] = torch.exp(-(torch.arange(N, device="cuda") % 5).float() / 4.0) if case["weighted"] else None
        s["scale"] = 1.0 / N
    elif op == "embed":
        s["E"] = _normal(g, (case["V"], case["D"]), 0.02, TYPES[case["type"]])
        s["idx"] = _tokens(g, case["N"], case["V"], case["pad"])
        s["scale"] = math.sqrt(case["D"])
        s["out"] = torch.zeros((case["N"], case["ld"]), dtype=TYPES[case["type"]], device="cuda")[:, :case["D"]]
    elif op == "embed_grad":
        s["dout"] = _normal(g, (case["N"], case["ld"]), 1.0, TYPES[case["type"]])[:, :case["D"]]
        s["idx"] = _tokens(g, case["N"], case["V"], case["pad"])
        s["scale"] = math.sqrt(case["D"])
        shape = (case["V"], case["D"])
        # the gradient that this one is added to
        s["base"] = _normal(g, shape, 1.0, TYPES[case["out"]]) if case["add"] else None
        s["dE"] = torch.zeros(shape, dtype=TYPES[case["out"]], device="cuda")
    else:
        sizes = _sizes(case)
        kinds = [("bf16", "f32")[i % 3 == 2] if case["type"] == "mixed" else case["type"] for i in range(len(sizes))]
        s["flat"], s["flat_out"], s["grads"], s["outs"] = {}, {}, [None] * len(sizes), [None] * len(sizes)
        for kind in sorted(set(kinds)):
            mine = [i for i in range(len(sizes)) if kinds[i] == kind]
            flat = torch.zeros(sum(_up(sizes[i], 8) for i in mine), dtype=TYPES[kind], device="cuda")
            out, at = torch.zeros_like(flat), 0
            for i in mine:
                s["grads"][i] = flat[at:at + sizes[i]].normal_(0.0, 10.0 ** (-1 - i % 3), generator=g)
                s["outs"][i] = out[at:at + sizes[i]]
                at += _up(sizes[i], 8)
            s["flat"][kind], s["flat_out"][kind] = flat, out
        s["max_norm"] = case["max_norm"]
    if own:
        from speculative_decoding_head_gb300 import binding
        if op == "ce":
            s["op"] = binding.LinearCE(N, K, V, layout=case["layout"])
            s["res"] = s["op"].new_outputs(dx="x" in case["grad"], dw="w" in case["grad"])
        elif op == "embed":
            s["op"] = binding.Embedding(case["N"], case["V"], case["D"])
        elif op == "embed_grad":
            s["op"] = binding.Embedding(case["N"], case["V"], case["D"])
        else:
            s["op"] = binding.GradClip(s["grads"], s["outs"])
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return (_run_own if own else _run_plain)(s, s["case"])


def _run_own(s, case):
    op = case["op"]
    if op == "ce":
        r = s["op"].forward(s["X"], s["W"], s["target"], U=s["U"], out=s["res"])
        if case["grad"]:
            s["op"].grad(s["X"], s["W"], s["target"], r["lse"], wt=s["wt"], scale=s["scale"], U=s["U"], out=r)
        return {k: r[k] for k in ("loss", "lse", "dX", "dW") if k in r}
    if op == "embed":
        return s["op"].lookup(s["E"], s["idx"], scale=s["scale"], out=s["out"])
    if op == "embed_grad":
        return s["op"].grad(s["dout"], s["idx"], scale=s["scale"], base=s["base"], out=s["dE"])
    norm = s["op"].clip(s["max_norm"])
    return {"norm": norm, "out": s["flat_out"]}


def _run_plain(s, case):
    op = case["op"]
    if op == "ce":
        X, W = s["X"].float(), s["W"].float()
        if case["layout"] == "kv":
            W = W.t()
        z = X @ W.t()
        if s["U"] is not None:
            z = z + s["U"]
        m = z.amax(1, keepdim=True)
        lse = m[:, 0] + torch.log(torch.exp(z - m).sum(1))
        t = s["target"].long()
        live = t >= 0
        t0 = t.clamp(min=0)
        zt = z.gather(1, t0[:, None])[:, 0]
        r = {"loss": torch.where(live, lse - zt, torch.zeros_like(lse)), "lse": lse}
        if case["grad"]:
            w = s["wt"] if s["wt"] is not None else torch.ones_like(lse)
            w = torch.where(live, w * s["scale"], torch.zeros_like(w))
            G = torch.exp(z - lse[:, None])
            G[torch.arange(t0.numel(), device=t0.device), t0] -= 1.0
            G = G * w[:, None]
            if "x" in case["grad"]:
                r["dX"] = (G @ W).to(BF16)
            if "w" in case["grad"]:
                r["dW"] = (X.t() @ G if case["layout"] == "kv" else G.t() @ X).to(BF16)
        return r
    if op == "embed":
        i = s["idx"].long()
        rows = s["E"][i.clamp(min=0)].float() * s["scale"]
        return torch.where((i >= 0)[:, None], rows, torch.zeros_like(rows)).to(TYPES[case["type"]])
    if op == "embed_grad":
        i = s["idx"].long()
        rows = s["dout"].float() * s["scale"]
        rows = torch.where((i >= 0)[:, None], rows, torch.zeros_like(rows))
        acc = s["base"].float() if case["add"] else torch.zeros((case["V"], case["D"]), dtype=F32, device="cuda")
        return acc.index_add(0, i.clamp(min=0), rows).to(TYPES[case["out"]])
    # every flat buffer holds nothing but gradients and zeros between them
    total = torch.zeros((), dtype=F32, device="cuda")
    for kind in s["flat"]:
        x = s["flat"][kind].float()
        total = total + (x * x).sum()
    norm = torch.sqrt(total)
    coef = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    return {"norm": norm, "out": {k: (x.float() * coef).to(x.dtype) for k, x in s["flat"].items()}}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "ce":
        N, K, V = case["N"], case["K"], case["V"]
        mats = 1 + len(case["grad"])
        byte = 2 * N * K + 2 * K * V + 4 * N + 8 * N + (4 * N * V if case["U"] else 0)
        byte += (4 * N if case["grad"] and case["weighted"] else 0)
        byte += (2 * N * K if "x" in case["grad"] else 0) + (2 * K * V if "w" in case["grad"] else 0)
        return {"bytes": byte, "flops": 2 * mats * N * K * V}
    if op == "embed":
        b = 2 if case["type"] == "bf16" else 4
        # a padded row reads nothing; a row looked up twice is read once at the least
        rows = min(case["N"] * (1 - case["pad"]), _distinct(case["N"] * (1 - case["pad"]), case["V"]))
        return {"bytes": int(b * case["D"] * (rows + case["N"]) + 4 * case["N"]), "flops": case["N"] * case["D"]}
    if op == "embed_grad":
        b, o = (2 if case[k] == "bf16" else 4 for k in ("type", "out"))
        rows = case["N"] * (1 - case["pad"])
        # every row of dE is written once; where another gradient is added, all of that is read too
        return {"bytes": int(b * case["D"] * rows + 4 * case["N"] + o * case["V"] * case["D"] * (2 if case["add"] else 1)),
                "flops": int(2 * rows * case["D"])}
    per = {"bf16": 2.0, "f32": 4.0, "mixed": 8.0 / 3.0}[case["type"]]
    # read once for the norm, read once more and written when the norm is known
    return {"bytes": int(3 * per * case["total"]), "flops": 3 * case["total"]}


def _distinct(n, V):
    """Tokens seen in n draws with frequencies that fall as 1 / rank (expected number, summed over octaves of the rank)."""
    got, lo = 0.0, 1.0
    while lo <= V:
        hi = min(2.0 * lo, V + 1.0)
        p = math.log(hi / lo) / math.log(V + 1) / (hi - lo)
        got += (hi - lo) * (1 - (1 - min(1.0, p)) ** n)
        lo = hi
    return got


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    op = case["op"]
    if op == "ce" and case["N"] * case["K"] * case["V"] * 2.0 * (1 + len(case["grad"])) > 8e12:
        return None
    s = prepare(case, seed)
    if op == "ce":
        return _exact_ce(case, s)
    if op == "embed":
        out = torch.zeros((case["N"], case["D"]), dtype=torch.float64, device="cuda")
        has = torch.nonzero(s["idx"] >= 0)[:, 0]
        out[has] = s["E"].index_select(0, s["idx"][has]).double() * s["scale"]
        return out
    if op == "embed_grad":
        if case["V"] * case["D"] * 8 > 6e9:
            return None
        # rows sorted by token, then the differences of a running sum at the ends of each token's run
        order = torch.argsort(s["idx"], stable=True)
        tok = s["idx"][order].long()
        order, tok = order[tok >= 0], tok[tok >= 0]
        out = s["base"].double() if case["add"] else torch.zeros((case["V"], case["D"]), dtype=torch.float64, device="cuda")
        if tok.numel() == 0:
            return out
        seen, runs = torch.unique_consecutive(tok, return_counts=True)
        ends = torch.cumsum(runs, 0)
        for c in range(0, case["D"], 128):
            run = torch.cumsum(s["dout"][order, c:c + 128].double(), 0)
            part = run[ends - 1]
            part[1:] -= run[ends[:-1] - 1]
            out[seen, c:c + 128] += part * s["scale"]
        return out
    total = sum(float(torch.linalg.vector_norm(x.double()).square()) for x in s["grads"])
    norm = math.sqrt(total)
    coef = min(1.0, s["max_norm"] / (norm + 1e-6))
    return {"norm": torch.tensor(norm, dtype=torch.float64), "out": {k: x.double() * coef for k, x in s["flat"].items()}}


def _exact_ce(case, s):
    """Row by row blocks, so that the 64-bit logits of a block alone are held."""
    N, V = case["N"], case["V"]
    W = s["W"].double() if case["layout"] == "kv" else s["W"].double().t()   # [K, V]
    loss, lse = (torch.zeros(N, dtype=torch.float64, device="cuda") for _ in range(2))
    dX = torch.zeros((N, case["K"]), dtype=torch.float64, device="cuda")
    dW = torch.zeros_like(W) if "w" in case["grad"] else None
    block = max(1, min(N, (1 << 27) // V))
    for a in range(0, N, block):
        b = min(N, a + block)
        X = s["X"][a:b].double()
        z = X @ W
        if s["U"] is not None:
            z += s["U"][a:b].double()
        logp = torch.log_softmax(z, 1)
        t = s["target"][a:b].long()
        live = torch.nonzero(t >= 0)[:, 0]
        lse[a:b] = (z - logp)[:, 0]
        loss[a + live] = -logp[live, t[live]]
        if case["grad"]:
            w = torch.zeros(b - a, dtype=torch.float64, device="cuda")
            w[live] = (s["wt"][a:b].double()[live] if s["wt"] is not None else 1.0) * s["scale"]
            p = torch.exp(logp) * w[:, None]
            p[live, t[live]] -= w[live]
            if "x" in case["grad"]:
                dX[a:b] = p @ W.t()
            if dW is not None:
                dW += X.t() @ p
    r = {"loss": loss, "lse": lse}
    if "x" in case["grad"]:
        r["dX"] = dX
    if dW is not None:
        r["dW"] = dW if case["layout"] == "kv" else dW.t()
    return r
