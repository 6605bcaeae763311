"""Cases for the operators that serve an output layer held in 4 bits and draw from its logits, with their plain forms.

quant       rows of a matrix into microscaled 4-bit floating point (e2m1 values, a scale per block of
            a row), given back here as the values that the 4 bits stand for. "mxfp4": blocks of 32, the
            scale a power of two. "nvfp4": blocks of 16, the scale e4m3, and a power of two per row.
rows        rows of such a matrix looked up by token, as values.
linear      z = X W^T (+ U) of a layer over the vocabulary whose W is held in 4 bits and whose X is
            brought into them within the call; sums of exact products.
sample      one token per row of logits from given uniform numbers, after temperature, top-k, top-p
            and min-p, with the log-probability that it was drawn with.
logprobs    the whole distribution that `sample` draws from, as log-probabilities (-inf where a token
            is left out): what a lossless verify of drafts reads as its target.

`own` false: elementary torch operations, in 64 bits where a value next to a border decides.
`own` true: the calls of speculative_decoding_head_gb300.binding.
"""

import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
TYPES = {"bf16": BF16, "f32": F32}
BLOCK = {"nvfp4": 16, "mxfp4": 32}
MASKED = -1e29                        # logits at or below this belong to tokens that are masked
LARGEST_QUANT = 129280 * 4096         # values of the largest matrix that is quantised
LARGEST_ROWS = 262144 * 256           # values of the largest lookup
LARGEST_LINEAR = 4096 * 5376 * 129280 # N K V of the largest product
LARGEST_LOGITS = 768 * 129280         # logits of the largest batch


def listed():
    return [
        # the hidden states of a decode batch (128 requests) on their way into the output layer
        {"name": "quant_states", "op": "quant", "R": 128, "K": 5120, "fmt": "nvfp4", "type": "bf16"},
        # an output matrix brought into 4 bits when a model is loaded
        {"name": "quant_matrix", "op": "quant", "R": 129280, "K": 4096, "fmt": "nvfp4", "type": "bf16"},
        # the Markov rows W1[x_{k-1}] of a round's 128 requests out of a table in 4 bits
        {"name": "rows_round", "op": "rows", "N": 128, "D": 256, "V": 129280, "fmt": "mxfp4", "out": "bf16", "pad": 0.0},
        # the same over a long teacher-forced batch, positions without a token among them
        {"name": "rows_long", "op": "rows", "N": 262144, "D": 256, "V": 129280, "fmt": "nvfp4", "out": "bf16", "pad": 0.1},
        # one request, one position: the output matrix streams by once
        {"name": "linear_one", "op": "linear", "N": 1, "K": 5120, "V": 129280, "fmt": "nvfp4", "out": "f32", "U": False},
        # the Markov bias of a round's 640 positions on their parallel logits
        {"name": "linear_markov", "op": "linear", "N": 640, "K": 256, "V": 129280, "fmt": "mxfp4", "out": "f32", "U": True},
        # the parallel logits of a round (128 requests x 5 positions)
        {"name": "linear_round", "op": "linear", "N": 640, "K": 5120, "V": 129280, "fmt": "nvfp4", "out": "f32", "U": False},
        # a long batch of positions scored at once
        {"name": "linear_long", "op": "linear", "N": 4096, "K": 5376, "V": 129280, "fmt": "nvfp4", "out": "bf16", "U": False},
        # the smallest round's two requests: latency
        {"name": "sample_tiny", "op": "sample", "N": 2, "V": 1024, "type": "f32", "set": "p", "shape": "flat", "requests": 0},
        # a decode batch, each request with settings of its own
        {"name": "sample_batch", "op": "sample", "N": 640, "V": 129280, "type": "bf16", "set": "mixed", "shape": "mixed",
         "requests": 0},
        # target rows of a small round, top-k and top-p together
        {"name": "logprobs_small", "op": "logprobs", "N": 192, "V": 32000, "type": "f32", "set": "kp", "shape": "mixed",
         "requests": 32},
        # the packed target rows of a whole round (128 requests, 6 rows each at the most) before their verify
        {"name": "logprobs_verify", "op": "logprobs", "N": 768, "V": 129280, "type": "f32", "set": "p", "shape": "mixed",
         "requests": 128},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant", "rows", "linear", "linear", "sample", "sample", "logprobs"])
    fmt = rng.choice(["nvfp4", "nvfp4", "mxfp4"])
    if op == "quant":
        while True:
            R, K = _log(rng, 1, 152000), _log(rng, 16, 6144)
            if R * K <= LARGEST_QUANT // 2:
                return {"op": op, "R": R, "K": K, "fmt": fmt, "type": rng.choice(["bf16", "bf16", "f32"])}
    if op == "rows":
        while True:
            N, D, V = _log(rng, 1, 262144), _log(rng, 16, 5120), _log(rng, 256, 152000)
            if N * D <= LARGEST_ROWS // 2 and V * D <= 4 * LARGEST_ROWS:
                return {"op": op, "N": N, "D": D, "V": V, "fmt": fmt, "out": rng.choice(["bf16", "f32"]),
                        "pad": rng.choice([0.0, 0.1])}
    if op == "linear":
        while True:
            N, K, V = _log(rng, 1, 4096), _log(rng, 16, 6144), _log(rng, 256, 152000)
            if N * K * V <= LARGEST_LINEAR:
                return {"op": op, "N": N, "K": K, "V": V, "fmt": fmt, "out": rng.choice(["f32", "f32", "bf16"]),
                        "U": rng.random() < 0.3}
    while True:
        N, V = _log(rng, 1, 2048), _log(rng, 256, 152000)
        if N * V <= LARGEST_LOGITS:
            break
    return {"op": op, "N": N, "V": V, "type": rng.choice(["f32", "f32", "bf16"]),
            "set": rng.choice(["p", "p", "k", "kp", "t", "minp", "mixed"]), "shape": rng.choice(["flat", "peaked", "mixed"]),
            "requests": rng.choice([0, max(1, N // rng.randint(1, 8))])}


# ---------------------------------------------------------------- inputs
def _up(x, m):
    return (x + m - 1) // m * m


def _normal(g, shape, std, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _rand(g, n, lo=0.0, hi=1.0):
    return torch.rand(n, generator=g, device="cuda") * (hi - lo) + lo


def _matrix(g, rows, cols, std, dtype):
    """Values of a common size, with channels that are a few times larger, as hidden states and weights have them."""
    x = _normal(g, (rows, cols), std, dtype)
    x[:, ::61] *= 6
    return x


def _tokens(g, n, V, pad):
    """Token ids with frequencies that fall as 1 / rank; a share `pad` of the rows holds none (-1)."""
    t = (torch.exp(torch.rand(n, generator=g, device="cuda", dtype=F64) * math.log(V + 1)) - 1).long().clamp_(0, V - 1)
    t = (t * 7919 + 12345) % V if V % 7919 else t
    return torch.where(torch.rand(n, generator=g, device="cuda") < pad, torch.full_like(t, -1), t).int()


def _logits(g, case):
    """Rows of logits: "flat" is the spread of the parallel logits alone, "peaked" has some hundred tokens that stand out
    of the rest, as a trained model's have. One in 128 tokens is masked, every other time by -inf or by the lowest value."""
    N, V, dtype = case["N"], case["V"], TYPES[case["type"]]
    z = _normal(g, (N, V), 2.0, F32)
    few = min(V, 200)
    lift = _rand(g, (N, few), 0.0, 1.0).square() * 12.0
    if case["shape"] == "flat":
        lift.zero_()
    elif case["shape"] == "mixed":
        lift[::2] = 0.0
    at = torch.randint(0, V, (N, few), generator=g, device="cuda")
    z.scatter_add_(1, at, lift)
    z = z.to(dtype)
    banned = torch.randint(0, V, (N, V // 128), generator=g, device="cuda")
    half = V // 256
    z.scatter_(1, banned[:, :half], -math.inf)
    z.scatter_(1, banned[:, half:], torch.finfo(dtype).min)
    return z


def _settings(g, kind, n):
    """temperature, top_k (0: off), top_p (1: off) and min_p (0: off) of n requests; None where the setting is not used."""
    T = _rand(g, n, 0.6, 1.2)
    k = torch.randint(1, 200, (n,), generator=g, device="cuda", dtype=torch.int32)
    p, mp = _rand(g, n, 0.7, 0.99), _rand(g, n, 0.01, 0.2)
    if kind == "t":
        return T, None, None, None
    if kind == "k":
        return T, k, None, None
    if kind == "p":
        return T, None, p, None
    if kind == "kp":
        return T, k, p, None
    if kind == "minp":
        return T, None, None, mp
    i = torch.arange(n, device="cuda") % 8
    T = torch.where(i == 0, torch.zeros_like(T), T)                    # greedy requests among the others
    k = torch.where((i == 1) | (i == 2), k, torch.zeros_like(k))
    p = torch.where((i >= 2) & (i <= 5), p, torch.ones_like(p))
    mp = torch.where((i == 5) | (i == 6), mp, torch.zeros_like(mp))
    return T, k, p, mp


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op == "quant":
        s["x"] = _matrix(g, case["R"], case["K"], 1.0, TYPES[case["type"]])
    elif op == "rows":
        s["E"] = _matrix(g, case["V"], case["D"], 0.02, BF16)
        s["idx"] = _tokens(g, case["N"], case["V"], case["pad"])
    elif op == "linear":
        N, K, V = case["N"], case["K"], case["V"]
        s["X"] = _matrix(g, N, K, 1.0, BF16)
        s["W"] = _matrix(g, V, K, 2.0 / math.sqrt(K), BF16)
        s["U"] = _normal(g, (N, _up(V, 4)), 2.0, F32)[:, :V] if case["U"] else None
    else:
        N, R = case["N"], case["requests"]
        s["z"] = _logits(g, case)
        s["u"] = _rand(g, N)
        s["set"] = _settings(g, case["set"], R or N)
        s["row_off"] = None
        if R:
            # the rows of request b are row_off[b] .. row_off[b + 1] - 1; the last row belongs to the last request
            cuts = torch.sort(torch.randint(0, N + 1, (R - 1,), generator=g, device="cuda"))[0]
            ends = torch.tensor([N], device="cuda")
            s["row_off"] = torch.cat([torch.zeros_like(ends), cuts, ends]).int()
    return s


def prepare(case, seed):
    s, op = _inputs(case, seed), case["op"]
    if own:
        from speculative_decoding_head_gb300 import binding
        if op == "quant":
            s["op"] = binding.Fp4Matrix(case["R"], case["K"], case["fmt"])
            s["out"] = torch.empty_like(s["x"])
        elif op == "rows":
            s["op"] = binding.Fp4Matrix(case["V"], case["D"], case["fmt"]).quantise(s.pop("E"))
        elif op == "linear":
            s["op"] = binding.Fp4Matrix(case["V"], case["K"], case["fmt"]).quantise(s.pop("W"))
            s["X4"] = binding.Fp4Matrix(case["N"], case["K"], case["fmt"])
            s["out"] = torch.empty((case["N"], _up(case["V"], 8)), dtype=TYPES[case["out"]], device="cuda")[:, :case["V"]]
        else:
            s["op"] = binding.Sampler(case["N"], case["V"], requests=case["requests"] or None)
            if op == "logprobs":
                s["out"] = torch.empty((case["N"], case["V"]), dtype=F32, device="cuda")
    elif op in ("rows", "linear"):
        # the matrix that is kept in 4 bits, as the values that it stands for (bf16 holds them)
        name = "E" if op == "rows" else "W"
        s[name] = _quantised(s[name], case["fmt"]).to(BF16)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return (_run_own if own else _run_plain)(s, s["case"])


def _run_own(s, case):
    op = case["op"]
    if op == "quant":
        return s["op"].quantise(s["x"]).lookup(out=s["out"])
    if op == "rows":
        return s["op"].lookup(s["idx"], dtype=TYPES[case["out"]])
    if op == "linear":
        return s["op"].linear(s["X4"].quantise(s["X"]), U=s["U"], out=s["out"])
    T, k, p, mp = s["set"]
    how = {"temperature": T, "top_k": k, "top_p": p, "min_p": mp, "row_off": s["row_off"]}
    if op == "sample":
        return s["op"].sample(s["z"], s["u"], **how)
    return s["op"].logprobs(s["z"], out=s["out"], **how)


def _run_plain(s, case):
    op = case["op"]
    if op == "quant":
        return _quantised(s["x"], case["fmt"]).to(s["x"].dtype)
    if op == "rows":
        i = s["idx"].long()
        rows = s["E"][i.clamp(min=0)].float()
        return torch.where((i >= 0)[:, None], rows, torch.zeros_like(rows)).to(TYPES[case["out"]])
    if op == "linear":
        z = _quantised(s["X"], case["fmt"]).float() @ s["W"].float().t()
        return (z if s["U"] is None else z + s["U"]).to(TYPES[case["out"]])
    x, w, kept = _distribution(s, case)
    w = torch.where(kept, w, torch.zeros_like(w))
    total = w.sum(1)
    if op == "logprobs":
        return torch.where(kept, x - torch.log(total)[:, None], torch.full_like(x, -math.inf)).float()
    c = torch.cumsum(w, 1)
    t = torch.searchsorted(c, (s["u"].double() * total)[:, None], right=True).clamp(max=case["V"] - 1)
    return {"token": t[:, 0].int(), "logp": (x.gather(1, t)[:, 0] - torch.log(total)).float()}


def _quantised(x, fmt):
    """The values that x [R, K] in 4 bits stands for, in 64 bits (they have few bits; what decides a rounding is x over a scale)."""
    R, K = x.shape
    B = BLOCK[fmt]
    x = torch.nn.functional.pad(x, (0, -K % B)).double().view(R, -1, B)
    top = x.abs().amax(2, keepdim=True)
    if fmt == "mxfp4":
        # 2^(floor(log2 of the largest) - 2): 4 and 6 are the largest values' octave
        scale = _two_to((torch.frexp(top)[1] - 3).clamp(-127, 127))
    else:
        # the row's power of two: the least with which the largest scale, largest / 6, is at most 448
        m, e = torch.frexp(top.amax(1, keepdim=True) / 2688.0)
        f = _two_to(torch.where(m == 0.5, e - 1, e).clamp(-100, 127))
        f = torch.where(m == 0, torch.ones_like(f), f)
        scale = _rounded(top / (6.0 * f), 3, -6, 448.0) * f
    q = _rounded(x / torch.where(scale == 0, torch.ones_like(scale), scale), 1, 0, 6.0)
    return (q * scale).view(R, -1)[:, :K]


def _rounded(x, bits, least, most):
    """x to the nearest number with `bits` bits behind its leading one (to the even one halfway), exponents from `least` on, at most `most`."""
    e = (torch.frexp(x)[1] - 1).clamp(min=least)
    step = _two_to(e - bits)
    return (torch.round(x / step) * step).clamp(-most, most)


def _two_to(e):
    """2^e in 64 bits, made of its bits (pow and exp2 may be off by some)."""
    return (e.long() + 1023 << 52).view(F64)


def _distribution(s, case):
    """x = (z - max) / T and e^x of every token in 64 bits, and which tokens are kept."""
    z = s["z"].float()
    N, V = z.shape
    z = torch.where(z <= MASKED, torch.full_like(z, -math.inf), z)
    T, k, p, mp = (None if v is None else v if s["row_off"] is None else v[_request(s["row_off"], N)] for v in s["set"])
    one = torch.ones(N, dtype=F64, device=z.device)
    T = one if T is None else T.double()
    k = torch.zeros_like(one).long() if k is None else k.long()
    p = one if p is None else p.double()
    mp = 0 * one if mp is None else mp.double()
    greedy = T == 0
    T, k = torch.where(greedy, one, T), torch.where(greedy, torch.ones_like(k), k)
    k = torch.where(k <= 0, torch.full_like(k, V), k)
    x = (z.double() - z.amax(1, keepdim=True).double()) / T[:, None]
    w = torch.exp(x)
    order = torch.sort(z, dim=1, descending=True, stable=True)[1]          # ties: the lowest token first
    ws = w.gather(1, order)
    ws = torch.where(torch.arange(V, device=z.device) < k[:, None], ws, torch.zeros_like(ws))
    before = torch.cumsum(ws, 1) - ws
    keep = (before < (p * ws.sum(1))[:, None]) | (p == 1)[:, None]
    keep &= torch.arange(V, device=z.device) < k[:, None]
    keep[:, 0] = True
    kept = torch.zeros_like(keep).scatter_(1, order, keep)
    kept &= (x * T[:, None] >= (T * torch.log(mp))[:, None]) & (z > -math.inf)
    return x, w, kept


def _request(row_off, N):
    return torch.searchsorted(row_off, torch.arange(N, device=row_off.device, dtype=torch.int32), right=True) - 1


# ---------------------------------------------------------------- what a pass cannot do without
def _held(rows, K, fmt):
    """Bytes of a matrix in 4 bits: half a byte a value, a byte a block, and nvfp4's 4 bytes a row."""
    return rows * (K / 2 + -(-K // BLOCK[fmt])) + (4 * rows if fmt == "nvfp4" else 0)


def work(case):
    op = case["op"]
    if op == "quant":
        b = 2 if case["type"] == "bf16" else 4
        return {"bytes": 2 * b * case["R"] * case["K"], "flops": 4 * case["R"] * case["K"]}
    if op == "rows":
        N = case["N"] * (1 - case["pad"])
        o = 2 if case["out"] == "bf16" else 4
        return {"bytes": int(_held(_distinct(N, case["V"]), case["D"], case["fmt"]) + o * case["N"] * case["D"] + 4 * case["N"]),
                "flops": int(N * case["D"])}
    if op == "linear":
        N, K, V = case["N"], case["K"], case["V"]
        o = 2 if case["out"] == "bf16" else 4
        return {"bytes": int(2 * N * K + _held(V, K, case["fmt"]) + (o + (4 if case["U"] else 0)) * N * V), "flops": 2 * N * K * V}
    b = 2 if case["type"] == "bf16" else 4
    out = 4 * case["N"] * case["V"] if op == "logprobs" else 8 * case["N"]
    return {"bytes": int(b * case["N"] * case["V"] + out + 16 * case["N"]), "flops": 4 * case["N"] * case["V"]}


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
def _nearest(x, grid):
    """The nearest member of a grid of magnitudes, of two as near the one at an even place."""
    a = x.abs().clamp(max=float(grid[-1]))
    hi = torch.searchsorted(grid, a).clamp(min=1, max=grid.numel() - 1)
    lo = hi - 1
    down, up = a - grid[lo], grid[hi] - a
    pick = torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return torch.sign(x) * grid[pick]


def _exact_values(x, fmt):
    """Block by block along a row, by the lists of numbers that 4 and 8 bits can hold."""
    e2m1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=F64, device="cuda")
    e4m3 = torch.tensor([m / 512.0 for m in range(8)] + [2.0 ** (e - 10) * (8 + m) for e in range(1, 16) for m in range(8)],
                        dtype=F64, device="cuda")[:127]
    out = torch.zeros(x.shape, dtype=F64, device="cuda")
    B = BLOCK[fmt]
    if fmt == "nvfp4":
        rowmax = x.abs().amax(1).double()
        f = _two_to(torch.ceil(torch.log2(rowmax.clamp(min=2.0 ** -149) / 2688.0)).clamp(min=-100))
        f = torch.where(f / 2 * 2688.0 >= rowmax, f / 2, f)
        f = torch.where(f * 2688.0 < rowmax, f * 2, f)
        f = torch.where(rowmax == 0, torch.ones_like(f), f)
    for c in range(0, x.shape[1], B):
        v = x[:, c:c + B].double()
        top = v.abs().amax(1)
        if fmt == "nvfp4":
            scale = _nearest(top / f / 6.0, e4m3) * f
        else:
            e = torch.floor(torch.log2(top.clamp(min=2.0 ** -149)))
            e = e - (_two_to(e) > top).double() + (_two_to(e + 1) <= top).double()
            scale = _two_to((e - 2).clamp(min=-127))
        safe = torch.where(scale == 0, torch.ones_like(scale), scale)
        out[:, c:c + B] = _nearest(v / safe[:, None], e2m1) * scale[:, None]
    return out


def exact(case, seed):
    op = case["op"]
    if op == "linear" and 2 * case["N"] * case["K"] * case["V"] > 5e12:
        return None
    s = _inputs(case, seed)
    if op == "quant":
        return _exact_values(s["x"], case["fmt"])
    if op == "rows":
        out = torch.zeros((case["N"], case["D"]), dtype=F64, device="cuda")
        has = torch.nonzero(s["idx"] >= 0)[:, 0]
        seen, where = torch.unique(s["idx"][has], return_inverse=True)
        out[has] = _exact_values(s["E"].index_select(0, seen), case["fmt"])[where]
        return out
    if op == "linear":
        X = _exact_values(s["X"], case["fmt"])
        out = torch.empty((case["N"], case["V"]), dtype=F64, device="cuda")
        for v in range(0, case["V"], 16384):
            out[:, v:v + 16384] = X @ _exact_values(s["W"][v:v + 16384], case["fmt"]).t()
        return out if s["U"] is None else out + s["U"].double()
    rows = [_exact_row(s, n) for n in range(case["N"])]
    if op == "logprobs":
        return torch.stack([logp for logp, _ in rows])
    tokens = torch.stack([t for _, t in rows])
    return {"token": tokens.int(), "logp": torch.stack([logp[t] for logp, t in rows])}


def _exact_row(s, n):
    """Log-probabilities of one row and the token drawn from them: thresholds over its distinct values, with the room
    left at the last of them given to the lowest tokens."""
    z = s["z"][n].double()
    z = torch.where(z <= MASKED, torch.full_like(z, -math.inf), z)
    b = n if s["row_off"] is None else int(torch.nonzero(s["row_off"] <= n)[-1])
    T, k, p, mp = (d if v is None else float(v[b]) for v, d in zip(s["set"], (1.0, 0, 1.0, 0.0)))
    if T == 0.0:
        T, k = 1.0, 1
    top = z.max()
    values, inverse, counts = torch.unique(z, return_inverse=True, return_counts=True)
    values, counts = values.flip(0), counts.flip(0)
    inverse = values.numel() - 1 - inverse
    w = torch.exp((values - top) / T)
    room = counts.clone()                                              # how many of each value's tokens are kept
    if k > 0:
        room = torch.minimum(room, (int(k) - (torch.cumsum(counts, 0) - counts)).clamp(min=0))
    if p < 1.0:
        mass = w * room
        before = torch.cumsum(mass, 0) - mass
        fit = torch.ceil((p * mass.sum() - before) / w).clamp(min=0)
        fit[0] = max(float(fit[0]), 1.0)
        room = torch.minimum(room, torch.nan_to_num(fit, posinf=0.0).clamp(max=float(z.numel())).long())
    if mp > 0.0:
        room = torch.where(values - top >= T * math.log(mp), room, torch.zeros_like(room))
    order = torch.argsort(inverse, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device="cuda")
    place -= (torch.cumsum(counts, 0) - counts)[inverse]               # a token's place among those of its value
    kept = (place < room[inverse]) & (z > -math.inf)
    p_kept = torch.where(kept, w[inverse], torch.zeros_like(z))
    total = p_kept.sum()
    logp = torch.where(kept, (z - top) / T - torch.log(total), torch.full_like(z, -math.inf))
    drawn = torch.nonzero(torch.cumsum(p_kept, 0) > s["u"][n].double() * total)[0, 0]
    return logp, drawn
