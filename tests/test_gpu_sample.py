"""Sampling and its distribution against sorting in 64 bits.

Tokens and the set of kept tokens are compared for equality: masses are taken to 2^-31 of
themselves, so a border is missed only where 64 bits come within about 1e-9 of it (none of these
draws does). Log-probabilities are (z - max) / T - log(mass) in fp32: the difference, 1 / T, their product and
the logarithm are each off by half a step, the mass by 2^-24 in fp32 and 2^-31 before, so by
2^-24 (3 |x| + 2 + |log mass|), and half a step of the sum."""

import math

import numpy as np
import pytest
import torch

import serve_ref as ref
from speculative_decoding_head_gb300.binding import DsparkError, Sampler

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
KINDS = ("none", "t", "k", "p", "kp", "minp", "all", "greedy")


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def logits(N, V, dtype, seed=0, std=2.0, masked=True):
    g = gen(seed)
    z = torch.empty(N, V, device="cuda").normal_(0.0, std, generator=g)
    if N > 1:  # every other row has tokens that stand out
        few = min(V, 50)
        at = torch.randint(0, V, (N, few), generator=g, device="cuda")
        lift = torch.rand(N, few, generator=g, device="cuda") * 10
        lift[::2] = 0
        z.scatter_add_(1, at, lift)
    z = z.to(dtype)
    if masked and V > 8:
        at = torch.randint(0, V, (N, V // 8), generator=g, device="cuda")
        z.scatter_(1, at[:, ::2], -math.inf)
        z.scatter_(1, at[:, 1::2], torch.finfo(dtype).min)
    return z


def check(z, how, u, row=None, sampler=None):
    """All of a batch's rows through both calls against the reference; row[n] is the entry of row n's settings."""
    N, V = z.shape
    T, k, p, mp = how
    s = sampler or Sampler(N, V)
    kw = dict(temperature=T, top_k=k, top_p=p, min_p=mp)
    got = s.sample(z, u, **kw)
    dist = s.logprobs(z, **kw)
    assert s.device_status() == 0
    tok, logp, dist = got["token"].cpu(), got["logp"].double().cpu().numpy(), dist.cpu()
    for n in range(N):
        one = {"T": T, "k": k, "p": p, "mp": mp}
        one = {a: float(b[n]) for a, b in one.items() if b is not None}
        t, lp, near = ref.row_sample(z[n], u[n], **one)
        assert int(tok[n]) == t, (n, int(tok[n]), t, near, one)
        with np.errstate(over="ignore"):  # below fp32's range the output is -inf
            want = ref.row_logprobs(z[n], **one)
            want = np.where(np.isfinite(want.astype(np.float32)), want, -np.inf)
        have = dist[n].double().numpy()
        assert np.array_equal(np.isfinite(have), np.isfinite(want)), (n, one, int(np.isfinite(have).sum()),
                                                                      int(np.isfinite(want).sum()))
        fine = np.isfinite(want)
        if t < 0:
            assert logp[n] == -math.inf
            continue
        x = np.abs(want[fine] - want[fine].max())
        tol = 2.0 ** -24 * (3 * x + 2 + abs(want[fine].max()) + np.abs(want[fine]))
        assert (np.abs(have[fine] - want[fine]) <= tol).all(), (n, one)
        assert abs(logp[n] - lp) <= 2.0 ** -24 * (4 * abs(lp) + 2 + 4 * abs(want[fine].max()))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("N,V", [(1, 1), (5, 2), (9, 31), (7, 512), (6, 513), (12, 1000), (40, 4097), (9, 32000)])
def test_against_sorting(N, V, kind, dtype):
    g = gen(V + N)
    z = logits(N, V, dtype, seed=V)
    check(z, ref.settings(kind, N, g), torch.rand(N, generator=g, device="cuda"))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", ("none", "k", "p", "all"))
@pytest.mark.parametrize("N,V", [(1, 129280), (20, 129280), (170, 50257), (3, 151936)])
def test_vocabularies(N, V, kind, dtype):
    g = gen(V + N)
    z = logits(N, V, dtype, seed=V)
    check(z, ref.settings(kind, N, g), torch.rand(N, generator=g, device="cuda"))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", ("none", "k", "p", "all"))
def test_large_parts_of_a_cluster(kind, dtype):
    """Sixteen CTAs that hold some 40000 (fp32) or 62500 (bf16) tokens each."""
    V = 600001 if dtype == F32 else 1000001
    g = gen(V)
    check(logits(2, V, dtype, seed=3), ref.settings(kind, 2, g), torch.rand(2, generator=g, device="cuda"))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_vocabularies_past_shared_memory(dtype):
    V = (1 << 21) + 77
    g = gen(1)
    z = logits(2, V, dtype, seed=1)
    for kind in ("none", "kp", "p", "all"):
        check(z, ref.settings(kind, 2, g), torch.rand(2, generator=g, device="cuda"))
    # many equal logits among them: the search by bits, and by index
    z = (z * 2).round() / 2
    for kind in ("k", "p"):
        check(z, ref.settings(kind, 2, g), torch.rand(2, generator=g, device="cuda"))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [100, 5000, 70000])
def test_equal_logits(V, dtype):
    g = gen(V)
    rows = [torch.zeros(V), torch.full((V,), -3.25), torch.arange(V) % 2 * 1.0, torch.arange(V) % 7 * 0.5,
            -(torch.arange(V) // 3 % 100) * 0.125, torch.where(torch.arange(V) % 5 == 0, -math.inf, 0.0),
            torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0)]
    z = torch.stack(rows).to("cuda", dtype)
    N = len(rows)
    u = torch.rand(N, generator=g, device="cuda")
    full = lambda v, t=F32: torch.full((N,), v, device="cuda", dtype=t)  # noqa: E731
    check(z, (None, None, None, None), u)
    for k in (1, 3, V // 2, V - 1, V, V + 9):
        check(z, (None, full(k, torch.int32), None, None), u)
    for p in (0.0, 1e-6, 0.3, 0.5, 0.9, 0.999999):
        check(z, (full(0.7), None, full(p), None), u)
    check(z, (full(0.0), full(50, torch.int32), full(0.5), full(0.5)), u)
    check(z, (full(1.3), full(V // 3, torch.int32), full(0.6), full(1.0)), u)


def test_ends_of_the_settings():
    N, V = 12, 3001
    z = logits(N, V, F32, seed=2)
    g = gen(2)
    u = torch.rand(N, generator=g, device="cuda")
    u[0], u[1], u[2], u[3] = 0.0, 1.0 - 2.0 ** -24, 2.0 ** -149, 2.0 ** -30
    full = lambda v, t=F32: torch.full((N,), v, device="cuda", dtype=t)  # noqa: E731
    for T in (1e-30, 1e-6, 0.01, 50.0, 1e6, 3e38):
        check(z, (full(T), None, full(0.9), None), u)
        check(z, (full(T), full(7, torch.int32), None, full(0.9)), u)
    for p in (2.0 ** -149, 1e-30, 0.5, 1.0 - 2.0 ** -24, 1.0):
        check(z, (None, None, full(p), None), u)
    for mp in (2.0 ** -149, 1e-30, 1e-3, 1.0 - 2.0 ** -24, 1.0):
        check(z, (full(0.8), None, None, full(mp)), u)
    for k in (-5, 0, 1, V - 1, V, 2 ** 31 - 1):
        check(z, (None, full(k, torch.int32), full(0.97), None), u)


def test_far_values():
    V = 2000
    z = torch.zeros(6, V, device="cuda")
    z[0] = torch.linspace(-1e28, 1e28, V)
    z[1] = torch.linspace(1e30, 3e38, V)
    z[2], z[2, 100] = -8e28, 5.0
    z[3] = torch.linspace(0, 1e-38, V)
    z[4] = 1e6 + torch.linspace(0, 30, V)
    z[5] = torch.finfo(F32).min
    z[5, 1234] = -9e28
    g = gen(3)
    u = torch.rand(6, generator=g, device="cuda")
    for kind in KINDS:
        check(z, ref.settings(kind, 6, g), u)


@pytest.mark.parametrize("V", [129280, (1 << 21) + 77])
def test_draws_among_the_lightest_tokens(V):
    """u below what one of the light tokens holds, and some of theirs: 2^-46.5 of the maximum's mass each."""
    light = -46.5 * math.log(2.0)
    z = torch.full((4, V), light, device="cuda")
    z[:, V - 1] = 0.0
    z[1::2, :700] = -math.inf
    u = torch.tensor([0.0, 0.0, 1e-12, 0.5], device="cuda")
    out = {"token": torch.full((4,), -7, device="cuda", dtype=torch.int32), "logp": torch.full((4,), 9.0, device="cuda")}
    Sampler(4, V).sample(z, u, out=out)
    tok = out["token"].tolist()
    # u S is less than one token's mass, and in the third row less than a hundred tokens'
    assert tok[0] == 0 and tok[1] == 700 and 0 <= tok[2] <= 200 and tok[3] == V - 1
    want = torch.tensor([light, light, light, 0.0], device="cuda") - math.log1p(V * 2.0 ** -46.5)
    assert ((out["logp"] - want).abs() <= 2.0 ** -22 * (1 + want.abs())).all()


@pytest.mark.parametrize("octaves", [20.5, 30.5, 36.5, 40.5, 44.5, 46.5])
@pytest.mark.parametrize("V", [129280, (1 << 21) + 77, 1 << 24])
def test_masses_of_many_light_tokens(V, octaves):
    """One heavy token and V - 1 light ones, whose mass together is 1 / 2 of its own down to 1e-14: the
    logarithm, and the top-p border in the middle of them, to 2e-10 of the mass."""
    z = torch.full((1, V), -octaves * math.log(2.0), device="cuda")
    z[0, V // 3] = 0.0
    m = math.exp(float(z[0, 0]))
    S = 1.0 + (V - 1) * m
    s = Sampler(1, V)
    lp = s.logprobs(z)
    for at, x in ((V // 3, 0.0), (0, float(z[0, 0])), (V - 1, float(z[0, 0]))):
        # half a step each of the mass in fp32, its logarithm and the result, and the light tokens' product
        assert abs(float(lp[0, at]) - (x - math.log(S))) <= 2.0 ** -24 * (3 + 2 * abs(x)) + 2e-10
    p = float(torch.tensor((1.0 + 0.5 * (V - 1) * m) / S, dtype=F32))
    if p < 1.0:
        kept = s.logprobs(z, top_p=torch.tensor([p], device="cuda")) > -math.inf
        n = int(kept.sum())
        want = 1 + max(0, math.ceil((p * S - 1.0) / m))
        assert abs(n - want) <= 1 + 2e-10 * S / m
        light = kept[0].clone()
        assert bool(light[V // 3])
        light[V // 3] = False
        first = int(light.sum())
        assert bool(light[:first + (first > V // 3)].sum() == first)  # the lowest of the light ones
    # Draws on both sides of the heavy token. Sums of 512 tokens are multiples of 2^-q of the mass, off by half a unit
    # each (equal sums all the same way), and in one of them so is each of 512 tokens.
    q = min(46, 62 - (V - 1).bit_length())
    off = 2e-10 + V * 2.0 ** -(q + 10) + 2.0 ** (8 - q)
    u = torch.tensor([(V // 3) * m / S * f for f in (0.0, 0.5)] + [((V // 3) * m + 0.5) / S], device="cuda")
    tok = Sampler(3, V).sample(z.expand(3, V).contiguous(), u)["token"].tolist()
    for t, x in zip(tok, u.double().tolist()):
        c = x * S
        want = math.floor(c / m) if c < (V // 3) * m else V // 3
        assert abs(t - want) <= 1 + off * S / m and (want == V // 3) == (t == V // 3)


def test_masks_next_to_the_maximum():
    """Temperatures so high that a masked token's finite logit would have a mass beside a maximum of -9e28."""
    V = 600
    z = torch.full((4, V), -1.00001e29, device="cuda")
    z[:, ::3] = -9.99e28
    z[:, 1::7] = -9.5e28
    g = gen(4)
    u = torch.rand(4, generator=g, device="cuda")
    T = torch.tensor([1e24, 1e26, 5e27, 1e30], device="cuda")
    check(z, (T, None, torch.full((4,), 0.7, device="cuda"), None), u)
    check(z, (T, torch.full((4,), 150, device="cuda", dtype=torch.int32), None, torch.full((4,), 0.5, device="cuda")), u)
    check(z, (T, None, None, None), u)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [3, 700, 40000])
def test_the_logarithm_next_to_one_kept_token(V, dtype):
    """A token that is kept alone has log-probability 0, one beside a light token that token's share to 2^-21 of it
    (two roundings of the sums, a division, the logarithm and the light token's mass: 2^-24 each at the most), and to
    2^-46: the sum and the token's own mass are multiples of 2^-46, half of that off each."""
    z = torch.empty(8, V, device="cuda").normal_(0.0, 0.5, generator=gen(V))
    z = (z - 60.0).to(dtype)
    z[torch.arange(8), torch.arange(8) * 7 % V] = torch.linspace(-9.0, 30.0, 8, device="cuda").to(dtype)
    u = torch.linspace(0.0, 0.99, 8, device="cuda")
    s, at = Sampler(8, V), torch.arange(8, device="cuda") * 7 % V
    full = lambda v, t=F32: torch.full((8,), v, device="cuda", dtype=t)  # noqa: E731
    for T in (0.7, 1.0, 1.9):
        for how in (dict(top_k=full(1, torch.int32)), dict(top_p=full(1e-3)), dict(min_p=full(0.5)),
                    dict(top_k=full(2, torch.int32), top_p=full(0.5))):
            got = s.sample(z, u, temperature=full(T), **how)
            lp = s.logprobs(z, temperature=full(T), **how)
            assert torch.equal(got["token"].long(), at) and (got["logp"] == 0).all()
            assert (lp.gather(1, at[:, None]) == 0).all() and torch.isfinite(lp).sum() == 8
    z = torch.full((1, V), -math.inf, device="cuda", dtype=dtype)
    z[0, 1], z[0, 2] = 1.5, -10.0
    for T in (0.5, 1.0, 2.0):
        lp = Sampler(1, V).logprobs(z, temperature=torch.tensor([T], device="cuda"))
        want = -math.log1p(math.exp(-11.5 / T))
        assert abs(float(lp[0, 1]) - want) <= 2.0 ** -21 * abs(want) + 2.0 ** -46


def test_many_kept_tokens():
    """top-k from the lists' limits on: as many tokens as threads, thousands, and nearly all."""
    N, V = 6, 40000
    z = logits(N, V, F32, seed=21)
    g = gen(21)
    u = torch.rand(N, generator=g, device="cuda")
    for k in (127, 128, 129, 256, 512, 640, 641, 1024, 3000, 30000):
        kk = torch.full((N,), k, device="cuda", dtype=torch.int32)
        check(z, (None, kk, torch.full((N,), 0.95, device="cuda"), None), u)
        check((z * 2).round() / 2, (None, kk, None, None), u)


def test_rows_with_nothing_left():
    V = 700
    z = logits(6, V, F32, seed=5)
    z[1], z[3] = -math.inf, torch.finfo(F32).min
    s = Sampler(6, V)
    p = torch.full((6,), 0.5, device="cuda")
    got = s.sample(z, torch.rand(6, generator=gen(5), device="cuda"), top_p=p)
    dist = s.logprobs(z, top_p=p, fill=-1e30)
    assert s.device_status() == 0
    for n in (1, 3):
        assert int(got["token"][n]) == -1 and float(got["logp"][n]) == -math.inf and (dist[n] == -1e30).all()
    assert (got["token"][[0, 2, 4, 5]] >= 0).all()
    have = dist[0].double().cpu().numpy()
    want = ref.row_logprobs(z[0], p=0.5)
    assert np.array_equal(have > -1e29, np.isfinite(want))


def test_rows_that_are_refused_on_the_device():
    V, N = 900, 14
    z = logits(N, V, F32, seed=6)
    z[0, 5], z[1, 899], z[2, 0] = float("nan"), float("inf"), float("nan")
    T, p, mp = (torch.full((N,), v, device="cuda") for v in (1.0, 0.9, 0.01))
    u = torch.full((N,), 0.3, device="cuda")
    T[3], T[4], T[5] = -1.0, float("nan"), float("inf")
    p[6], p[7] = -0.1, 1.5
    mp[8], mp[9] = 1.1, float("nan")
    u[10], u[11], u[12] = 1.0, -1e-9, float("nan")
    s = Sampler(N, V)
    got = s.sample(z, u, temperature=T, top_p=p, min_p=mp)
    assert s.device_status() == 4
    assert (got["token"][:13] == -1).all() and got["logp"][:13].isnan().all()
    t, _, _ = ref.row_sample(z[13], 0.3, p=float(p[13]), mp=float(mp[13]))
    assert int(got["token"][13]) == t
    s.reset()
    dist = s.logprobs(z, temperature=T, top_p=p, min_p=mp)
    assert s.device_status() == 4
    assert (dist[:10] == -math.inf).all() and (dist[10:].max(1)[0] > -math.inf).all()


@pytest.mark.parametrize("R,N", [(1, 9), (6, 20), (700, 300)])
def test_rows_of_requests(R, N):
    V = 1111
    g = gen(R)
    z = logits(N, V, F32, seed=7)
    first, end = 2, N - 3
    cuts = torch.sort(torch.randint(first, end + 1, (R - 1,), generator=g, device="cuda"))[0]
    off = torch.cat([torch.tensor([first], device="cuda"), cuts, torch.tensor([end], device="cuda")]).int()
    how = ref.settings("all", R, g)
    owner = torch.searchsorted(off, torch.arange(N, device="cuda", dtype=torch.int32), right=True) - 1
    mine = (owner >= 0) & (owner < R)
    each = [v[owner.clamp(0, R - 1)].contiguous() for v in how]
    u = torch.rand(N, generator=g, device="cuda")
    s, t = Sampler(N, V, requests=R), Sampler(N, V)
    names = ("temperature", "top_k", "top_p", "min_p")
    want, wdist = t.sample(z, u, **dict(zip(names, each))), t.logprobs(z, **dict(zip(names, each)))
    out = {"token": torch.full((N,), -7, dtype=torch.int32, device="cuda"), "logp": torch.full((N,), 7.0, device="cuda")}
    z[~mine] = float("nan")  # rows of no request are not read
    s.sample(z, u, row_off=off, out=out, **dict(zip(names, how)))
    dist = s.logprobs(z, row_off=off, out=torch.full((N, V), 7.0, device="cuda"), **dict(zip(names, how)))
    assert s.device_status() == 0
    assert torch.equal(out["token"][mine], want["token"][mine]) and torch.equal(out["logp"][mine], want["logp"][mine])
    assert torch.equal(dist[mine], wdist[mine])
    assert (out["token"][~mine] == -7).all() and (out["logp"][~mine] == 7).all() and (dist[~mine] == 7).all()


def test_strides_alignment_and_no_logp():
    N, V = 11, 4099
    for dtype in (F32, BF16):
        big = logits(2 * N, V + 13, dtype, seed=8)
        g = gen(8)
        u = torch.rand(N, generator=g, device="cuda")
        how = ref.settings("kp", N, g)
        for view in (big[:N, :V], big[::2, 1:1 + V], big[N:, 3:3 + V]):
            check(view, how, u)
            s = Sampler(N, V)
            kw = dict(zip(("temperature", "top_k", "top_p", "min_p"), how))
            a = s.sample(view, u, **kw)
            b = s.sample(view, u, out={"token": torch.empty(N, dtype=torch.int32, device="cuda")}, **kw)
            assert torch.equal(a["token"], b["token"])
            out = torch.full((N, V + 9), 7.0, device="cuda")
            s.logprobs(view, out=out[:, 5:5 + V], **kw)
            assert torch.equal(out[:, 5:5 + V], s.logprobs(view, **kw))
            assert (out[:, :5] == 7).all() and (out[:, 5 + V:] == 7).all()


def test_offsets_past_32_bits():
    N, V = 17000, 129280
    z = torch.empty(N, V, dtype=BF16, device="cuda").normal_(0.0, 2.0, generator=gen(9))
    u = torch.rand(N, generator=gen(10), device="cuda")
    p = torch.full((N,), 0.9, device="cuda")
    got = Sampler(N, V).sample(z, u, top_p=p)
    for n in (0, 16612, N - 1):
        t = Sampler(1, V).sample(z[n:n + 1], u[n:n + 1], top_p=p[:1])
        assert int(t["token"]) == int(got["token"][n]) and float(t["logp"]) == float(got["logp"][n])
        assert int(t["token"]) == ref.row_sample(z[n], u[n], p=float(p[0]))[0]


def test_frequencies():
    """Draws of one row follow its distribution: chi-squared over 40 kept tokens, 2^20 draws (39 degrees of freedom;
    the value 120 has a probability below 1e-9)."""
    V, n = 40, 1 << 20
    z = logits(1, V, F32, seed=11, std=1.0, masked=False)
    u = torch.rand(n, generator=gen(12), device="cuda")
    got = Sampler(n, V).sample(z.expand(n, V).contiguous(), u)["token"]
    have = torch.bincount(got.long(), minlength=V).double().cpu().numpy()
    kept, w = ref.row_distribution(z[0])
    want = w / w.sum() * n
    assert ((have - want) ** 2 / want).sum() < 120


def test_streams_and_graphs():
    N, V = 30, 9000
    z, u = logits(N, V, F32, seed=13), torch.rand(N, generator=gen(13), device="cuda")
    p = torch.full((N,), 0.8, device="cuda")
    s = Sampler(N, V)
    want = s.sample(z, u, top_p=p)
    wdist = s.logprobs(z, top_p=p)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, dist = s.sample(z, u, top_p=p, stream=side), s.logprobs(z, top_p=p, stream=side)
    side.synchronize()
    assert torch.equal(got["token"], want["token"]) and torch.equal(dist, wdist)
    g = torch.cuda.CUDAGraph()
    out = {k: torch.empty_like(v) for k, v in want.items()}
    with torch.cuda.graph(g):
        s.sample(z, u, top_p=p, out=out)
        s.logprobs(z, top_p=p, out=dist)
    z.copy_(logits(N, V, F32, seed=14))
    u.copy_(torch.rand(N, generator=gen(14), device="cuda"))
    g.replay()
    torch.cuda.synchronize()
    again = s.sample(z, u, top_p=p)
    assert torch.equal(again["token"], out["token"]) and torch.equal(again["logp"], out["logp"])
    assert torch.equal(dist, s.logprobs(z, top_p=p)) and not torch.equal(out["token"], want["token"])


def test_refusals():
    with pytest.raises(DsparkError):
        Sampler(4, 0)
    with pytest.raises(DsparkError):
        Sampler(-1, 5)
    with pytest.raises(DsparkError):
        Sampler(4, 5, requests=0)
    s = Sampler(4, 64)
    z, u = torch.zeros(4, 64, device="cuda"), torch.zeros(4, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    for bad in (z.half(), z[:, :32], z[:3], z.cpu(), torch.zeros(64, 4, device="cuda").t()):
        with pytest.raises(DsparkError):
            s.sample(bad, u)
        with pytest.raises(DsparkError):
            s.logprobs(bad)
    for kw in (dict(temperature=u[:3]), dict(top_k=u), dict(top_p=u.double()), dict(min_p=u.cpu()), dict(row_off=off)):
        with pytest.raises(DsparkError):
            s.sample(z, u, **kw)
    with pytest.raises(DsparkError):
        s.sample(z, u[:2])
    for rows in (z[:1].expand(4, 64), torch.zeros(300, device="cuda").as_strided((4, 64), (63, 1))):
        with pytest.raises(DsparkError):  # rows that overlap
            s.sample(rows, u)
        with pytest.raises(DsparkError):
            s.logprobs(z, out=rows)
    with pytest.raises(DsparkError):
        s.logprobs(z, out=z)
    with pytest.raises(DsparkError):
        s.logprobs(z, out=torch.zeros(4, 64, device="cuda", dtype=BF16))
    assert Sampler(0, 64).sample(z[:0], u[:0])["token"].shape == (0,)
