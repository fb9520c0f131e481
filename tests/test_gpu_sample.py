"""Sampling and unmasking on the GPU against the float64 oracle. Tokens have to be equal. A log-probability is
x - m - log(sum e^(x - m)): the sum's relative error is below 2^-17 (sample.cuh bounds it by 4e-6 < 2^-17), one rounding
of the result to fp32 adds 2^-24 of it."""
import math

import numpy as np
import pytest
import torch

from oracle import answer_oracle as ao

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bd():
    import block_diffusion_lm_bdlm_gb300 as m

    m.load_library()
    return m


DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def logits_of(seed, rows, vocab, dtype, *, sharp=4.0, head=0, pad=0, masked=0.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, vocab)) * sharp * np.exp2(rng.uniform(-2, 0, (rows, 1)))
    for r in range(rows):
        if head:
            x[r, rng.integers(0, vocab, head)] += 12 + 2 * rng.standard_normal(head)
    x[rng.random((rows, vocab)) < masked] = -np.inf
    buf = torch.full((rows, vocab + pad), 1e4, dtype=dtype, device="cuda")  # what lies between rows would win
    buf[:, :vocab] = torch.from_numpy(x).to(dtype).cuda()
    return buf[:, :vocab]


def at(x, i):
    return x[i].item() if isinstance(x, torch.Tensor) else torch.tensor(x, dtype=torch.float32).item()


def check(bd, x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    token, lp = bd.bdlm_sample(x, u, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)
    token, lp = token.cpu().numpy(), lp.double().cpu().numpy()
    host, uh = x.double().cpu().numpy(), u.double().cpu().numpy()
    for i in range(x.shape[0]):
        want, wlp = ao.sample_row(host[i], uh[i], at(temperature, i), at(top_k, i), at(top_p, i), at(min_p, i))
        assert token[i] == want, (i, token[i], want)
        if want < 0:
            assert lp[i] == -np.inf
        else:
            assert abs(lp[i] - wlp) <= 2.0 ** -17 + 2.0 ** -24 * abs(wlp), (i, lp[i], wlp)


HOW = [dict(), dict(temperature=0.7), dict(temperature=0.0), dict(top_k=1), dict(top_k=7), dict(top_k=50, temperature=1.3), dict(top_p=0.9),
       dict(top_p=0.3, temperature=0.5), dict(min_p=0.05), dict(min_p=0.4, temperature=2.0), dict(top_k=40, top_p=0.95, min_p=0.02, temperature=0.8),
       dict(top_p=0.999), dict(top_p=0.0), dict(min_p=1.0), dict(top_k=300, top_p=0.5)]


@pytest.mark.parametrize("how", HOW, ids=lambda h: "-".join(f"{k}{v}" for k, v in h.items()) or "plain")
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab,pad", [(1, 0), (2, 1), (7, 0), (65, 3), (513, 0), (4099, 5)])
def test_small(bd, dtype, vocab, pad, how):
    x = logits_of(vocab, 9, vocab, DTYPES[dtype], pad=pad, head=min(3, vocab))
    u = torch.rand(9, generator=torch.Generator("cuda").manual_seed(vocab), device="cuda")
    check(bd, x, u, **how)


@pytest.mark.parametrize("how", [HOW[i] for i in (0, 1, 4, 6, 8, 10, 11, 14)], ids=lambda h: "-".join(f"{k}{v}" for k, v in h.items()) or "plain")
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab,pad,sharp,head", [(32001, 0, 3.0, 20), (50257, 3, 1.0, 0), (131072, 0, 6.0, 40), (262144, 8, 0.2, 0)])
def test_large(bd, dtype, vocab, pad, sharp, head, how):
    rows = 6 if vocab < 60000 else 3
    x = logits_of(vocab + 1, rows, vocab, DTYPES[dtype], pad=pad, sharp=sharp, head=head, masked=0.2)
    u = torch.rand(rows, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    check(bd, x, u, **how)


def test_many_rows_of_every_kind(bd):
    """A parameter for each row, many more rows than fit at once."""
    rows, vocab = 1500, 3001
    x = logits_of(5, rows, vocab, torch.bfloat16, head=8, pad=1)
    rng = np.random.default_rng(6)
    f = lambda v: torch.tensor(v, dtype=torch.float32, device="cuda")
    check(bd, x, f(rng.random(rows)), temperature=f(rng.choice([0.0, 1.0, 0.6, 1.7], rows)),
          top_k=torch.tensor(rng.choice([0, 1, 20, 3000, 5000, -4], rows), dtype=torch.int32, device="cuda"),
          top_p=f(rng.choice([1.0, 0.9, 0.2, 1.5, 0.0], rows)), min_p=f(rng.choice([0.0, 0.1, -1.0, 3.0], rows)))


@pytest.mark.parametrize("dtype", DTYPES)
def test_cuts_about_the_number_of_listed_tokens(bd, dtype):
    """top-k from below the parts that a row is looked at in to above what a list holds, with and without the other cuts, in rows
    that several CTAs share: all of them must take the same way."""
    ks = [31, 32, 33, 63, 64, 65, 100, 119, 120, 121, 127, 128, 129, 200, 255, 256, 257, 400, 511, 512, 513, 800]
    x = logits_of(21, len(ks), 140001, DTYPES[dtype], pad=3, head=10)
    u = torch.rand(len(ks), generator=torch.Generator("cuda").manual_seed(2), device="cuda")
    k = torch.tensor(ks, dtype=torch.int32, device="cuda")
    for how in (dict(), dict(min_p=0.02), dict(min_p=1e-4, temperature=1.5), dict(top_p=0.9), dict(top_p=0.99, min_p=0.3)):
        check(bd, x, u, top_k=k, **how)


@pytest.mark.parametrize("dtype", DTYPES)
def test_equal_logits(bd, dtype):
    """Every border is hit exactly: u, p and k at whole numbers of equal tokens."""
    vocab = 4096
    x = torch.full((8, vocab), 2.5, dtype=DTYPES[dtype], device="cuda")
    u = torch.tensor([0.0, 0.25, 0.5, 0.75, 1.0, 1.0 / 4096, 4095.0 / 4096, 0.3], device="cuda")
    for how in (dict(), dict(top_k=1024), dict(top_p=0.5), dict(top_k=2048, top_p=0.25), dict(min_p=1.0), dict(top_k=4096), dict(top_k=4095),
                dict(top_p=2.0 ** -12), dict(temperature=0.0)):
        check(bd, x, u, **how)
    x[:, ::2] = 1.5  # two values: the cut lies among equal ones of either
    for how in (dict(top_k=3000), dict(top_k=2048), dict(top_p=0.9), dict(top_p=0.8, temperature=1e6), dict(top_p=0.99, temperature=0.01)):
        check(bd, x, u, **how)


@pytest.mark.parametrize("dtype", DTYPES)
def test_logits_that_are_no_numbers(bd, dtype):
    t, inf, nan, low = DTYPES[dtype], math.inf, math.nan, torch.finfo(DTYPES[dtype]).min
    rows = [[-inf] * 40, [nan] * 40, [-inf, nan] * 20, [0.0, inf] * 20, [nan, inf, -inf, 1.0] * 10, [low] * 40, [low, -inf] * 20,
            [low] * 39 + [5.0], [-0.0, 0.0] * 20, [torch.finfo(t).max, low] * 20, [nan] * 39 + [low], [1e-30, -1e-30] * 20]
    x = torch.tensor(rows).to(t).cuda()
    for vocab in (40, 39):
        for how in (dict(), dict(temperature=0.0), dict(top_k=3), dict(top_p=0.5), dict(min_p=0.5), dict(top_k=30, top_p=0.9, min_p=0.1), dict(top_k=39)):
            for u in (0.0, 0.37, 1.0):
                check(bd, x[:, :vocab], torch.full((len(rows),), u, device="cuda"), **how)


def test_extreme_parameters(bd):
    x = logits_of(11, 6, 700, torch.float32)
    for u in (-1.0, 2.0, 0.5):
        uu = torch.full((6,), u, device="cuda")
        for how in (dict(temperature=1e-5), dict(temperature=1e-7), dict(temperature=-1.0), dict(temperature=math.nan), dict(temperature=1e20),
                    dict(temperature=3e38), dict(top_p=1e-30), dict(top_p=1 - 2.0 ** -24), dict(top_p=math.nan), dict(min_p=1e-38),
                    dict(min_p=math.nan), dict(top_k=2 ** 31 - 1), dict(top_k=-2 ** 31), dict(top_k=699), dict(top_p=-1.0)):
            check(bd, x, uu, **how)


@pytest.mark.parametrize("dtype", DTYPES)
def test_cold_rows_of_equal_logits(bd, dtype):
    """More equal logits than a list holds, at temperatures at which every other value of the type is many octaves away."""
    x = torch.full((4, 9000), -3.0, dtype=DTYPES[dtype], device="cuda")
    x[:, 5::9] = 2.0
    x[2, 7] = 2.015625
    u = torch.tensor([0.1, 0.5, 0.9, 1.0], device="cuda")
    for t in (1e-5, 3e-6, 1e-3, 0.03):
        for how in (dict(), dict(top_k=600), dict(top_p=0.5), dict(min_p=0.3), dict(top_k=700, top_p=0.7, min_p=0.9)):
            check(bd, x, u, temperature=t, **how)


def test_rows_with_their_token_are_left(bd):
    x = logits_of(3, 50, 1000, torch.bfloat16)
    x[1::3] = math.nan
    now = torch.full((50,), 7, dtype=torch.int32, device="cuda")
    now[1::3] = 11
    u = torch.rand(50, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    want, wlp = bd.bdlm_sample(x, u)
    out, lp = torch.full_like(now, -5), torch.full((50,), 3.25, device="cuda")
    bd.bdlm_sample(x, u, tokens=now, mask_id=7, out=out, logprob=lp)
    todo = now == 7
    assert torch.equal(out, torch.where(todo, want, -5)) and torch.equal(lp, torch.where(todo, wlp, 3.25))
    bd.bdlm_sample(x, u, tokens=now, mask_id=7, out=now, logprob=lp)  # in place
    assert torch.equal(now, torch.where(todo, want, 11))
    with pytest.raises(ValueError):
        bd.bdlm_sample(x, u, tokens=now, mask_id=7)


def test_captured_and_on_another_stream(bd):
    x = logits_of(8, 33, 9001, torch.float16, pad=1)
    u = torch.rand(33, device="cuda")
    want = bd.bdlm_sample(x, u, top_p=0.8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = bd.bdlm_sample(x, u, top_p=0.8, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    out, lp = torch.empty_like(want[0]), torch.empty_like(want[1])
    with torch.cuda.graph(graph):
        bd.bdlm_sample(x, u, top_p=0.8, out=out, logprob=lp)
    u.copy_(torch.rand(33, device="cuda"))
    x.copy_(logits_of(9, 33, 9001, torch.float16))
    graph.replay()
    want = bd.bdlm_sample(x, u, top_p=0.8)
    assert torch.equal(out, want[0]) and torch.equal(lp, want[1])


def test_logprobs_near_0(bd):
    """A token that has nearly all of the weight: its log-probability is -log(1 + rest), and the rest, summed apart from
    it, is good to kQuick = 4e-6 of itself (sample.cuh); the logarithm and its rounding add 2^-22."""
    rng = np.random.default_rng(3)
    for dtype in DTYPES.values():
        x = torch.from_numpy(rng.standard_normal((40, 3000))).to(dtype).cuda()
        x[:, 77] = torch.linspace(9, 17, 40).to(dtype).cuda()
        for how in (dict(temperature=0.0), dict(top_k=1), dict(top_p=0.1), dict(min_p=0.9), dict()):
            token, lp = bd.bdlm_sample(x, torch.full((40,), 0.5, device="cuda"), **how)
            for i in range(40):
                want, wlp = ao.sample_row(x[i].double().cpu().numpy(), 0.5, **how)
                assert token[i].item() == want == 77 and abs(lp[i].item() - wlp) <= (4e-6 + 2.0 ** -22) * abs(wlp), (how, i)


def test_no_rows(bd):
    token, lp = bd.bdlm_sample(torch.zeros((0, 5), device="cuda"), torch.zeros(0, device="cuda"))
    assert token.shape == lp.shape == (0,)


def test_sample_refusals(bd):
    x, u = torch.zeros((4, 8), device="cuda"), torch.zeros(4, device="cuda")
    for kw in (dict(u=u[:3]), dict(u=u.double()), dict(temperature=u[:2]), dict(top_k=u), dict(tokens=u), dict(out=u), dict(top_k=2 ** 31),
               dict(mask_id=2 ** 31), dict(logprob=torch.zeros(4)), dict(x=x.t()), dict(x=x.double()), dict(x=x[0]), dict(x=x[:, :0]),
               dict(x=x[:1].expand(4, 8))):
        args = {"x": x, "u": u}
        args.update({k: kw[k] for k in ("x", "u") if k in kw})
        with pytest.raises(ValueError):
            bd.bdlm_sample(args["x"], args["u"], **{k: v for k, v in kw.items() if k not in ("x", "u")})


# ----------------------------------------------------------------- unmasking
def blocks(seed, rows, masked=0.6):
    rng = np.random.default_rng(seed)
    T = int(sum(rows)) + 5
    tokens = np.where(rng.random(T) < masked, 77, rng.integers(0, 50, T))
    sampled = np.where(rng.random(T) < 0.1, -1, rng.integers(100, 200, T))
    lp = -np.round(rng.random(T) * 8) / 8  # many equal ones
    lp[rng.random(T) < 0.05] = np.nan
    lp[rng.random(T) < 0.05] = -np.inf
    lp[rng.random(T) < 0.05] = -0.0
    return tokens, sampled, lp, np.concatenate([[0], np.cumsum(rows)])


@pytest.mark.parametrize("rows", [[1], [32] * 16, [0, 5, 1, 0, 33, 256, 257, 7], [1023, 1024, 1025, 2], [5000, 3], list(range(90))], ids=str)
@pytest.mark.parametrize("per", ["n", "threshold", "both"])
def test_unmask(bd, rows, per):
    tokens, sampled, lp, off = blocks(len(rows), rows)
    rng = np.random.default_rng(4)
    n = len(rows)
    i32 = lambda v: torch.as_tensor(np.asarray(v)).to("cuda", torch.int32)
    f32 = lambda v: torch.as_tensor(np.asarray(v)).to("cuda", torch.float32)
    k = rng.integers(-1, 20, n) if per != "threshold" else np.zeros(n, dtype=int)
    thr = rng.choice([-0.5, -0.125, 0.0, 1.0, -np.inf, np.nan], n) if per != "n" else np.full(n, np.nan)
    want, left = ao.unmask(tokens, sampled, lp.astype(np.float32), off, 77, k, thr)
    t = i32(tokens)
    out = torch.full_like(t, -9)
    got, gl = bd.bdlm_unmask(t, i32(sampled), f32(lp), i32(off), 77, n_min=i32(k) if per != "threshold" else 0,
                             threshold=f32(thr) if per != "n" else math.nan, out=out, check=True)
    assert got is out and np.array_equal(out.cpu().numpy()[:off[-1]], want[:off[-1]]) and torch.all(out[off[-1]:] == -9)
    assert np.array_equal(gl.cpu().numpy(), left)
    bd.bdlm_unmask(t, i32(sampled), f32(lp), i32(off), 77, n_min=i32(k), threshold=f32(thr), out=t, check=True)  # in place
    assert np.array_equal(t.cpu().numpy(), want)


def test_unmask_one_number_for_all(bd):
    tokens, sampled, lp, off = blocks(1, [40, 41])
    i32 = lambda v: torch.as_tensor(np.asarray(v)).to("cuda", torch.int32)
    want, left = ao.unmask(tokens, sampled, lp.astype(np.float32), off, 77, [6, 6], [-0.25, -0.25])
    got, gl = bd.bdlm_unmask(i32(tokens), i32(sampled), torch.as_tensor(lp).float().cuda(), i32(off), 77, n_min=6, threshold=-0.25)
    assert np.array_equal(got.cpu().numpy()[:81], want[:81]) and np.array_equal(gl.cpu().numpy(), left)


@pytest.mark.parametrize("off,bad", [([1, 3, 6], 0), ([0, 4, 3], 1), ([0, 3, 8], 1), ([0, -1, 5], 0)])
def test_unmask_malformed_offsets(bd, off, bad):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    t, out, left = i32([7] * 6), i32([-3] * 6), i32([-4, -4])
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    args = (t, i32([1] * 6), torch.zeros(6, device="cuda"), i32(off), 7)
    bd.bdlm_unmask(*args, n_min=1, out=out, left=left, workspace=ws)
    assert bd.bdlm_read_error(ws) == 6 and left[bad].item() == -4
    with pytest.raises(bd.BDLMError):
        bd.bdlm_unmask(*args, n_min=1, check=True)


def test_unmask_without_rows(bd):
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    out, left = bd.bdlm_unmask(e, e, torch.zeros(0, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda"), 7, check=True)
    assert out.numel() == 0 and left.tolist() == [0, 0, 0]
    with pytest.raises(bd.BDLMError):
        bd.bdlm_unmask(e, e, torch.zeros(0, device="cuda"), torch.ones(4, dtype=torch.int32, device="cuda"), 7, check=True)
