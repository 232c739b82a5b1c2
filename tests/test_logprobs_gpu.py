"""Log probabilities of given tokens, entropy, alternatives and the logits' gradient, against the
formulas in 64 bits.

Tolerances, in units of 2^-24 (half an fp32 step): u = (z - m) / T is off by three roundings (the
difference, 1 / T, the product), 3 |u|.  Each exponential then by 3 |u| + 4 (ex2: 2 ulp), weighted by
itself in every sum, and the sum by one unit for each of a thread's additions (a row's elements
over 256 threads, at most) and of the joins (below 32).  So ln S is off by slack = V / 256 + 40 + 4 E|u|,
a log probability by that and 4 (|u| + ln S) more, and the entropy by (1 + H + E|u|) slack.  The gradient's terms are
off by slack + 4 |ln p| times their magnitude (the exponent's two roundings), and the result by its own
rounding; fp16 results below 2^-14 by half their fixed step, 2^-25.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def g():
    import programming_tiled_gemm_gb300 as g
    return g


@pytest.fixture(scope="module")
def lib(g):
    lib = g.Gemm(0)
    yield lib
    assert lib.device_status() == g.GEMM_OK
    lib.close()


def make(seed, rows, V, dtype, ld=None, offset=0, scale=2.0):
    """logits in rows `ld` apart that start `offset` elements into their storage"""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ld = ld or V
    flat = torch.full((rows * ld + offset + 8,), float("nan"), device="cuda", dtype=dtype)
    logits = flat[offset:offset + rows * ld].view(rows, ld)[:, :V]
    logits.copy_((torch.randn(rows, V, generator=gen, device="cuda") * scale).to(dtype))
    tokens = torch.randint(0, V, (rows,), generator=gen, device="cuda")
    return logits, tokens


def reference(logits, tokens, temperature):
    """(u, logp, p, H, E|u|, ln S) in 64 bits; rows without a finite logit: logp -inf, H 0"""
    z = logits.double()
    m = z.amax(1, keepdim=True)
    u = (z - torch.where(m == -math.inf, torch.zeros_like(m), m)) / temperature
    e = torch.exp(u)
    s = e.sum(1, keepdim=True)
    logp = torch.where(s > 0, u - torch.log(s), torch.full_like(u, -math.inf))
    p = torch.where(s > 0, e / s, torch.zeros_like(e))
    h = -torch.where(p > 0, p * logp, torch.zeros_like(p)).sum(1)
    eu = torch.where(p > 0, -p * u, torch.zeros_like(p)).sum(1)
    return u, logp, p, h, eu, torch.where(s > 0, torch.log(s), torch.zeros_like(s))[:, 0]


def slack(V, eu):
    return U * (V / 256 + 40 + 4 * eu)


def check_forward(logits, tokens, temperature, top, r):
    rows, V = logits.shape
    u, logp, p, h, eu, ln_s = reference(logits, tokens, temperature)
    given = (tokens >= 0) & (tokens < V)
    at = torch.where(given, tokens, torch.zeros_like(tokens))[:, None]
    want = torch.where(given, logp.gather(1, at)[:, 0], torch.zeros_like(h))
    ut = u.gather(1, at)[:, 0].abs()
    sl = slack(V, eu)
    tol = sl + 4 * U * (torch.where(ut.isfinite(), ut, torch.zeros_like(ut)) + ln_s)
    # (equal where both are -inf; a value beyond fp32's range, lowest / 0.5, is -inf there)
    same = (r.logprobs == want.float()) | ((r.logprobs.double() - want).abs() <= tol)
    assert bool(same.all()), (r.logprobs, want)
    if r.entropy is not None:
        assert bool(((r.entropy.double() - h).abs() <= sl * (1 + h + eu)).all())
    m = logits.double().amax(1)
    assert torch.equal(r.stats[:, 0].double(), m)
    assert bool(((r.stats[:, 1].double() - ln_s).abs() <= sl + 4 * U * ln_s).all())
    if top:
        vals, order = torch.sort(logits.float(), dim=1, descending=True, stable=True)
        n = min(top, V)
        vals, order = vals[:, :n], order[:, :n]
        want_tok = torch.where(vals > -math.inf, order, torch.full_like(order, -1))
        assert torch.equal(r.top_tokens[:, :n], want_tok)
        assert bool((r.top_tokens[:, n:] == -1).all()) and bool((r.top_logprobs[:, n:] == -math.inf).all())
        lp = torch.where(want_tok >= 0, logp.gather(1, order), torch.full_like(logp[:, :n], -math.inf))
        ua = u.gather(1, order).abs()
        tol = sl[:, None] + 4 * U * (torch.where(ua.isfinite(), ua, torch.zeros_like(ua)) + ln_s[:, None])
        got = r.top_logprobs[:, :n].double()
        assert bool(((r.top_logprobs[:, :n] == lp.float()) | ((got - lp).abs() <= tol)).all())


def check_backward(logits, tokens, temperature, gain, dh, got):
    rows, V = logits.shape
    _, logp, p, h, eu, _ = reference(logits, tokens, temperature)
    given = (tokens >= 0) & (tokens < V)
    zero = torch.zeros(rows, device="cuda", dtype=torch.float64)
    gd = torch.where(given, gain.double(), zero) if gain is not None else zero
    hd = dh.double() if dh is not None else zero
    live = logp.amax(1) > -math.inf
    lp = torch.where(p > 0, logp, torch.zeros_like(logp))
    delta = torch.zeros_like(p).scatter_(1, torch.where(given, tokens, torch.zeros_like(tokens))[:, None], 1.0)
    delta *= (given & live).double()[:, None]
    want = (gd[:, None] * (delta - p) - hd[:, None] * p * (lp + h[:, None])) / temperature
    size = (gd.abs()[:, None] * (delta + p) + hd.abs()[:, None] * p * (lp.abs() + h[:, None])) / temperature
    fp32 = (slack(V, eu)[:, None] + 4 * U * lp.abs() + 8 * U) * size + 1e-38
    # ex2's results below 2^-126, the least normal number, are 0: up to that of p is lost
    fp32 += 2.0 ** -126 * ((gd.abs()[:, None] + hd.abs()[:, None] * (lp.abs() + h[:, None])) / temperature)
    # the entropy itself is off by its own tolerance, which p multiplies
    fp32 += hd.abs()[:, None] * p * (slack(V, eu) * (1 + h + eu))[:, None] / temperature
    dt = got.dtype
    tol = fp32 + want.abs() * (torch.finfo(dt).eps / 2) + (2.0 ** -25 if dt is torch.float16 else 0.0)
    bad = (got.double() - want).abs() > tol * (1 + 1e-6)
    assert not bool(bad.any()), (int(bad.sum()), got[bad][:5], want[bad][:5])


SHAPES = [(1, 1, None, 0), (3, 2, None, 0), (5, 7, None, 1), (2, 31, 37, 3), (4, 255, None, 5), (7, 1000, 1003, 1),
          (1, 32000, None, 0), (300, 257, None, 0), (64, 5003, 5008, 0), (3, 50257, None, 0), (2, 131072, None, 8),
          (1000, 1031, None, 0)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,V,ld,offset", SHAPES)
def test_forward_and_backward(lib, rows, V, ld, offset, dtype):
    logits, tokens = make(rows * V, rows, V, DTYPES[dtype], ld, offset)
    top = min(20, V + 2)
    r = lib.token_logprobs(logits, tokens, top=top, entropy=True)
    check_forward(logits, tokens, 1.0, top, r)
    gen = torch.Generator(device="cuda").manual_seed(7)
    gain, dh = torch.randn(rows, generator=gen, device="cuda"), torch.randn(rows, generator=gen, device="cuda")
    dl = lib.token_logprobs_backward(gain, logits, tokens, r, dentropy=dh)
    check_backward(logits, tokens, 1.0, gain, dh, dl)
    # into rows of another alignment, and over the logits themselves
    buf = torch.full((rows, V + 5), 3.0, device="cuda", dtype=DTYPES[dtype])
    into = lib.token_logprobs_backward(gain, logits, tokens, r, dentropy=dh, out=buf[:, 2:V + 2])
    assert torch.equal(into, dl) and bool((buf[:, :2] == 3).all()) and bool((buf[:, V + 2:] == 3).all())
    plain = lib.token_logprobs_backward(gain, logits, tokens, r)
    check_backward(logits, tokens, 1.0, gain, None, plain)
    lib.token_logprobs_backward(gain, logits, tokens, r, out=logits)
    assert torch.equal(logits, plain)


@pytest.mark.parametrize("top", [0, 1, 2, 31, 32])
@pytest.mark.parametrize("temperature", [0.05, 0.7, 1.0, 30.0])
def test_temperatures_and_tops(lib, temperature, top):
    logits, tokens = make(top + 3, 9, 4099, torch.float32)
    tokens[::2] = torch.tensor([-100, -1, 4099, 1 << 40, -(1 << 62)], device="cuda")
    r = lib.token_logprobs(logits, tokens, top=top, entropy=True, temperature=temperature)
    check_forward(logits, tokens, temperature, top, r)
    only = lib.token_logprobs(logits, tokens, top=top, temperature=temperature)
    assert only.entropy is None and torch.equal(only.logprobs, r.logprobs)
    gain, dh = torch.linspace(-2, 2, 9, device="cuda"), torch.linspace(1, -1, 9, device="cuda")
    for g_, h_ in ((gain, dh), (gain, None), (None, dh)):
        dl = lib.token_logprobs_backward(g_, logits, tokens, r, dentropy=h_, temperature=temperature)
        check_backward(logits, tokens, temperature, g_, h_, dl)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_equal_logits_go_by_the_lower_index(lib, dtype):
    """constant rows, few distinct values, rising and falling rows: every logit ties or is a new best"""
    V = 20011
    rows = torch.stack([torch.zeros(V), torch.full((V,), -3.0), torch.arange(V) % 7 * 1.0, -(torch.arange(V) % 3) * 1.0,
                        torch.arange(V) / V, -torch.arange(V) / V, (torch.arange(V) * 7919 % V) * 1.0,
                        torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0)]).to("cuda").to(DTYPES[dtype])
    tokens = torch.zeros(len(rows), dtype=torch.int64, device="cuda")
    for one in (False, True):  # all rows in one call, and a row a call (shared by more CTAs)
        for i in range(len(rows) if one else 1):
            l, t = (rows[i:i + 1], tokens[:1]) if one else (rows, tokens)
            r = lib.token_logprobs(l, t, top=32, entropy=True)
            check_forward(l, t, 1.0, 32, r)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("temperature", [0.5, 1.0])
def test_masked_logits(lib, dtype, temperature):
    """-inf, the type's lowest value, rows of either only, one left, a masked token given"""
    dt, V, low = DTYPES[dtype], 3001, torch.finfo(DTYPES[dtype]).min
    logits, tokens = make(5, 10, V, dt)
    tokens[:] = torch.arange(10, device="cuda") * 17
    logits[0] = -math.inf
    logits[1] = low
    logits[2, 1:] = -math.inf
    logits[3, :-1] = low
    logits[4, ::2] = -math.inf
    logits[5, 1::2] = low
    logits[6, tokens[6]] = -math.inf
    logits[7, tokens[7]] = low
    logits[8, 5:] = -math.inf
    logits[9] = -math.inf
    logits[9, 2999] = low
    r = lib.token_logprobs(logits, tokens, top=8, entropy=True, temperature=temperature)
    check_forward(logits, tokens, temperature, 8, r)
    assert r.entropy[0] == 0 and r.logprobs[0] == -math.inf and bool((r.top_tokens[0] == -1).all())
    assert not bool(r.entropy.isnan().any())
    gain, dh = torch.ones(10, device="cuda"), torch.full((10,), 0.5, device="cuda")
    dl = lib.token_logprobs_backward(gain, logits, tokens, r, dentropy=dh, temperature=temperature)
    assert bool((dl[0] == 0).all()) and not bool(dl.isnan().any())
    check_backward(logits[1:], tokens[1:], temperature, gain[1:], dh[1:], dl[1:])


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("place", [0, 1500, 3000])
def test_rows_with_nan_or_infinity(lib, value, entropy, place):
    logits, tokens = make(9, 4, 3001, torch.bfloat16)
    clean = lib.token_logprobs(logits, tokens, top=4, entropy=entropy)
    logits[1, place] = value
    logits[2] = value
    tokens[2] = -100
    r = lib.token_logprobs(logits, tokens, top=4, entropy=entropy)
    for a, b in zip(r, clean):
        if a is not None:
            assert torch.equal(a[[0, 3]], b[[0, 3]])
    assert r.logprobs[1].isnan() and r.logprobs[2] == 0
    assert bool((r.top_tokens[1:3] == -1).all()) and bool(r.top_logprobs[1:3].isnan().all())
    if entropy:
        assert bool(r.entropy[1:3].isnan().all())
    dl = lib.token_logprobs_backward(torch.ones(4, device="cuda"), logits, tokens, r)
    assert bool(dl[1].isnan().all()) and bool((dl[2] == 0).all()) and not bool(dl[[0, 3]].isnan().any())


def test_gradient_against_differences(lib):
    """(f(z + e) - f(z - e)) / 2 e of f = g . logprobs + h . entropy, in 64 bits from the library's own formula's
    definition: the gradient of what the forward call computes"""
    rows, V, t = 3, 11, 0.8
    logits, tokens = make(3, rows, V, torch.float32, scale=1.0)
    gain, dh = torch.tensor([1.0, -2.0, 0.5], device="cuda"), torch.tensor([0.3, 0.0, -1.0], device="cuda")
    r = lib.token_logprobs(logits, tokens, entropy=True, temperature=t)
    dl = lib.token_logprobs_backward(gain, logits, tokens, r, dentropy=dh, temperature=t)

    def f(z):
        lp = torch.log_softmax(z / t, 1)
        return (gain.double() * lp.gather(1, tokens[:, None])[:, 0] - dh.double() * (lp.exp() * lp).sum(1)).sum()

    e = 1e-5  # the difference's own error: e^2 f''' / 6 < 1e-9, and 1e-16 / e
    for i in range(rows):
        for j in range(V):
            z = logits.double()
            hi, lo = z.clone(), z.clone()
            hi[i, j] += e
            lo[i, j] -= e
            assert abs(float(dl[i, j]) - float((f(hi) - f(lo)) / (2 * e))) < 1e-5
    # and of the calls themselves: fp32 results a step of 1/64 apart; (1/64)^2 f''' / 6 < 2e-4, 2^-22 / (1/32) < 1e-5
    step = 1.0 / 64
    for i in range(rows):
        for j in range(0, V, 3):
            vals = []
            for s in (step, -step):
                z = logits.clone()
                z[i, j] += s
                o = lib.token_logprobs(z, tokens, entropy=True, temperature=t)
                vals.append(float((gain * o.logprobs + dh * o.entropy)[i]))
            assert abs(float(dl[i, j]) - (vals[0] - vals[1]) / (2 * step)) < 1e-3


def test_rows_without_a_gradient_are_not_read(lib):
    logits, tokens = make(4, 6, 999, torch.float16)
    r = lib.token_logprobs(logits, tokens, entropy=True)
    gain = torch.tensor([0.0, 1.0, 0.0, 1.0, 0.0, 1.0], device="cuda")
    tokens[3] = -100
    logits[0], logits[3] = math.nan, math.nan  # (stats are those of the clean rows)
    dl = lib.token_logprobs_backward(gain, logits, tokens, r)
    assert bool((dl[[0, 2, 3, 4]] == 0).all())
    check_backward(logits[[1, 5]], tokens[[1, 5]], 1.0, gain[[1, 5]], None, dl[[1, 5]])


def test_empty_streams_graphs_and_repeats(lib, g):
    r = lib.token_logprobs(torch.empty(0, 50, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), top=3,
                           entropy=True)
    assert r.top_tokens.shape == (0, 3) and r.stats.shape == (0, 2)
    logits, tokens = make(1, 40, 9001, torch.bfloat16)
    gain = torch.randn(40, device="cuda")
    want = lib.token_logprobs(logits, tokens, top=5, entropy=True)
    dwant = lib.token_logprobs_backward(gain, logits, tokens, want, dentropy=gain)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = lib.token_logprobs(logits, tokens, top=5, entropy=True)
        dother = lib.token_logprobs_backward(gain, logits, tokens, other, dentropy=gain)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = lib.token_logprobs(logits, tokens, top=5, entropy=True)
        dkept = lib.token_logprobs_backward(gain, logits, tokens, kept, dentropy=gain)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(want, other, kept):
            assert torch.equal(a, b) and torch.equal(a, c)
        assert torch.equal(dwant, dother) and torch.equal(dwant, dkept)


def test_offsets_past_32_bits(lib):
    """rows that lie more than 2^31 elements into the logits"""
    rows, V = 3, 1000
    ld = (1 << 30) + 24
    big = torch.empty(2 * ld + V, device="cuda", dtype=torch.bfloat16)
    logits = torch.as_strided(big, (rows, V), (ld, 1))
    src, tokens = make(2, rows, V, torch.bfloat16)
    logits.copy_(src)
    r = lib.token_logprobs(logits, tokens, top=3, entropy=True)
    check_forward(src, tokens, 1.0, 3, r)
    gain = torch.ones(rows, device="cuda")
    dl = lib.token_logprobs_backward(gain, logits, tokens, r, out=logits)
    check_backward(src, tokens, 1.0, gain, None, dl.contiguous())


def test_refusals(lib, g):
    logits, tokens = make(1, 4, 100, torch.bfloat16)
    ok = lib.token_logprobs(logits, tokens)
    for t in (0.0, -1.0, math.inf, math.nan, 1e-39):
        with pytest.raises(g.GemmError):
            lib.token_logprobs(logits, tokens, temperature=t)
        with pytest.raises(g.GemmError):
            lib.token_logprobs_backward(None, logits, tokens, ok, temperature=t)
    with pytest.raises(g.GemmError):
        lib.token_logprobs(logits, tokens, top=33)
    for bad in (tokens.int(), tokens[:3], tokens.cpu(), torch.zeros(8, dtype=torch.int64, device="cuda")[::2]):
        with pytest.raises(ValueError):
            lib.token_logprobs(logits, bad)
    with pytest.raises(ValueError):
        lib.token_logprobs(logits, tokens, top=-1)
    with pytest.raises(ValueError):
        lib.token_logprobs(logits.t(), tokens)
    with pytest.raises(ValueError):
        lib.token_logprobs(logits[:, :0], tokens)
    with pytest.raises(TypeError):
        lib.token_logprobs(logits.double(), tokens)
    with pytest.raises(ValueError):
        lib.token_logprobs_backward(None, logits, tokens, ok, dentropy=torch.ones(4, device="cuda"))
    with pytest.raises(TypeError):
        lib.token_logprobs_backward(None, logits, tokens, ok, out=logits.float())
    # the C entry's own checks (nothing is launched)
    f, p, n = g.token_logprobs, logits.data_ptr(), lib.launch_count()
    s = ok.stats.data_ptr()
    args = [lib.handle, 4, 100, p, 100, g.GEMM_BF16, tokens.data_ptr(), 1.0, s, None, s, 0, None, None]

    def call(**kw):
        a = list(args)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    assert call(_1=-1) == call(_2=0) == call(_3=None) == call(_4=99) == call(_5=7) == call(_6=None) == g.GEMM_ERR_INVALID_ARG
    assert call(_8=None) == call(_10=None) == call(_11=-1) == call(_11=2) == g.GEMM_ERR_INVALID_ARG
    assert call(_3=p + 1) == call(_6=tokens.data_ptr() + 4) == call(_8=s + 2) == g.GEMM_ERR_ALIGNMENT
    assert call(_2=(1 << 30) + 1, _4=1 << 31) == g.GEMM_ERR_UNSUPPORTED
    b = g.token_logprobs_backward
    assert b(lib.handle, 4, 100, p, 100, g.GEMM_BF16, tokens.data_ptr(), 1.0, s, None, s, s, p, 100) == g.GEMM_ERR_INVALID_ARG
    assert b(lib.handle, 4, 100, p, 100, g.GEMM_BF16, tokens.data_ptr(), 1.0, s, None, s, None, p, 104) == g.GEMM_ERR_INVALID_ARG
    assert lib.launch_count() == n
