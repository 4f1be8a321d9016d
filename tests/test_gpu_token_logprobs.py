"""GPU parity of token log-probs, entropy, top alternatives and their gradient against oracle/token_logprobs.py.

Tolerances: t_j is rounded once (2^-24 of |t|), the SFU exponential adds 2^-22 relative, sums of V <= 60000 terms in
fp32 trees of depth ~25 add ~2^-20 relative; entropy and log-probs are those errors times the size of the logs."""

import numpy as np
import pytest
import torch

import speculative_decoding_verification_72_gb300 as sv
from oracle import token_logprobs as L

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    sv.load_library()


def check(x, tokens, T=1.0, n_top=0):
    x = x.to(DEV)
    B, R, V = x.shape
    r = sv.spec_token_logprobs(x, torch.as_tensor(tokens, dtype=torch.int32, device=DEV), temperature=T, n_top=n_top)
    x64 = x.double().cpu().numpy().reshape(B * R, V)
    want = L.token_logprobs(x64, np.asarray(tokens).reshape(-1), T, n_top)
    size = 1 + np.abs(np.where(np.isfinite(x64), x64, 0)).max(1) / T + np.log(V)
    for k in ("logprob", "entropy", "lse"):
        got = r[k].double().cpu().numpy().reshape(-1)
        assert np.array_equal(np.isnan(got), np.isnan(want[k])), k
        fine = np.isfinite(want[k])
        assert np.array_equal(got[~fine], want[k][~fine], equal_nan=True), k
        assert (np.abs(got - want[k])[fine] <= (2.0 ** -20 * size)[fine]).all(), k
    assert np.array_equal(r["status"].cpu().numpy().reshape(-1), want["status"])
    if n_top:
        rows = ~np.isnan(want["lse"])
        assert np.array_equal(r["top_tokens"].cpu().numpy().reshape(-1, n_top)[rows], want["top_tokens"][rows])
        got = r["top_logprobs"].double().cpu().numpy().reshape(-1, n_top)
        inf = np.isinf(want["top_logprobs"])
        assert np.array_equal(np.isinf(got), inf) and np.array_equal(np.isnan(got), np.isnan(want["top_logprobs"]))
        ok = inf | np.isnan(got) | (np.abs(got - np.where(inf, 0, want["top_logprobs"])) <= 2.0 ** -20 * size[:, None])
        assert ok.all()
    return r, x64


@pytest.mark.parametrize("B,R,V,dtype,n_top,T", [
    (1, 1, 1, F32, 1, 1.0), (1, 1, 2, BF, 5, 1.0), (2, 3, 31, BF, 32, 0.7), (3, 2, 1003, F32, 20, 1.3),
    (2, 2, 16384, BF, 20, 1.0), (2, 2, 16385, BF, 7, 1.0), (1, 3, 8191, F32, 3, 0.5), (2, 5, 50257, BF, 20, 1.0),
    (1, 2, 40961, F32, 32, 1.0), (3, 1, 33, F32, 0, 1.0)])
def test_values(B, R, V, dtype, n_top, T):
    g = torch.Generator().manual_seed(V)
    x = (torch.randn((B, R, V), generator=g) * 3).to(dtype)
    check(x, torch.randint(-1, V, (B, R), generator=g).numpy(), T, n_top)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["equal", "two_values", "lowest", "one_left", "half_masked", "huge", "sorted", "zeros"])
def test_ties_masks_and_ranges(kind, dtype):
    V = 20001
    g = torch.Generator().manual_seed(5)
    x = torch.randn((1, 2, V), generator=g) * 3
    if kind == "equal":
        x[:] = 1.5
    elif kind == "two_values":
        x = (torch.rand(x.shape, generator=g) < 0.5).float()
    elif kind == "lowest":
        x[torch.rand(x.shape, generator=g) < 0.999] = torch.finfo(dtype).min
    elif kind == "one_left":
        x[:, :, :] = -float("inf")
        x[0, 0, 17000] = 2.0
        x[0, 1, 3], x[0, 1, 19999] = -1e30, -1e30
    elif kind == "half_masked":
        x[:, :, 3000:] = -float("inf")
    elif kind == "huge":
        x = x * 1e4
    elif kind == "sorted":
        x = x.sort(-1).values
    else:
        x = torch.where(torch.rand(x.shape, generator=g) < 0.5, 0.0, -0.0)
    check(x.to(dtype), [[17000, 2]], 1.0, 20)


@pytest.mark.parametrize("n_top", [1, 20, 32])
@pytest.mark.parametrize("left", [33, 500, 900, 4000])
def test_a_range_of_tokens_left(left, n_top):
    """All but a short range masked: few groups of threads have a maximum, and many elements reach their lowest."""
    V = 70001
    g = torch.Generator().manual_seed(left)
    x = torch.randn((1, 3, V), generator=g).to(BF)
    for r, at in enumerate((0, 16300, V - left)):
        x[0, r, :at], x[0, r, at + left:] = -float("inf"), -float("inf")
    check(x, [[0, 16300, 5]], 1.0, n_top)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_lowest_value_beside_masked_tokens(dtype):
    x = torch.full((1, 3, 9000), -float("inf"))
    low = torch.finfo(dtype).min
    x[0, 0, ::3] = low                  # the row's maximum is the lowest value
    x[0, 1, ::3], x[0, 1, 4001] = low, 1.0
    x[0, 2, ::2], x[0, 2, 1::4] = -0.0, low
    check(x.to(dtype), [[3, 0, 1]], 1.0, 6)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_that_are_not_finite(dtype):
    x = torch.randn((1, 6, 3000))
    x[0, 0, 7] = float("nan")
    x[0, 1, 2999] = float("inf")
    x[0, 2] = -float("inf")
    x[0, 3, :100] = -float("inf")
    x[0, 4, 0], x[0, 4, 1:] = float("nan"), -float("inf")
    r, x64 = check(x.to(dtype), [[1, -1, 5, 50, 0, 4000]], 1.0, 4)
    g = torch.ones((1, 6), device=DEV)
    d = sv.spec_token_logprobs_backward(x.to(dtype).to(DEV), torch.tensor([[1, -1, 5, 50, 0, 4000]], device=DEV), r["saved"], g, g)
    assert torch.isnan(d[0, [0, 1, 4]]).all() and (d[0, 2] == 0).all() and torch.isfinite(d[0, [3, 5]]).all()


@pytest.mark.parametrize("pad", [0, 1, 3, 8])
def test_strided_rows_and_odd_starts(pad):
    V = 5001
    g = torch.Generator().manual_seed(6)
    for dtype in (BF, F32):
        wide = (torch.randn((2, 3, V + pad + 1), generator=g) * 2).to(dtype).to(DEV)
        x = wide[:, :, pad:pad + V]
        tok = torch.randint(0, V, (2, 3), generator=g)
        r, x64 = check(x.cpu(), tok.numpy(), 1.0, 9)
        s = sv.spec_token_logprobs(x, tok.to(DEV), n_top=9)
        assert torch.equal(s["top_tokens"], r["top_tokens"])
        assert torch.allclose(s["logprob"], r["logprob"], atol=2.0 ** -19, rtol=0)
        check_grad(x, tok, 1.0, g)


def check_grad(x, tok, T, gen, out=None):
    B, R, V = x.shape
    g, h = torch.randn((B, R), generator=gen), torch.randn((B, R), generator=gen)
    x64 = x.double().cpu().numpy().reshape(-1, V)
    tok = tok.to(device=DEV, dtype=torch.int32)
    saved = sv.spec_token_logprobs(x, tok, temperature=T)["saved"]
    d = sv.spec_token_logprobs_backward(x, tok, saved, g.to(DEV), h.to(DEV), temperature=T, out=out)
    want = L.backward(x64, tok.cpu().numpy().reshape(-1), g.double().numpy().reshape(-1), h.double().numpy().reshape(-1), T)
    got = d.double().cpu().numpy().reshape(-1, V)
    # p and ln p as in the forward pass: relative 2^-20 of the size of the logs, and the type's rounding
    size = 1 + np.abs(np.where(np.isfinite(x64), x64, 0)).max(1, keepdims=True) / T + np.log(V)
    p = np.abs(want) + (np.abs(g).double().numpy().reshape(-1, 1) + np.abs(h).double().numpy().reshape(-1, 1) * size) * np.exp(
        np.where(np.isfinite(x64), x64, -np.inf) / T - L.token_logprobs(x64, np.full(B * R, -1), T)["lse"][:, None]) / T
    u = 2.0 ** -8 if x.dtype == BF else 2.0 ** -24
    assert (np.abs(got - want) <= u * np.abs(want) * 1.01 + 2.0 ** -19 * size * p + 1e-30).all()
    return d


@pytest.mark.parametrize("B,R,V,dtype,T", [(1, 1, 1, F32, 1.0), (2, 3, 33, BF, 0.7), (1, 2, 16385, BF, 1.0), (2, 2, 8193, F32, 1.3),
                                           (1, 3, 50257, BF, 1.0)])
def test_gradient(B, R, V, dtype, T):
    gen = torch.Generator().manual_seed(V)
    x = (torch.randn((B, R, V), generator=gen) * 3).to(dtype).to(DEV)
    if V > 100:
        x[0, 0, 5:50] = -float("inf")
    tok = torch.randint(-1, V, (B, R), generator=gen)
    d = check_grad(x, tok, T, gen)
    # another alignment than the logits', and over the logits
    odd = torch.empty(B * R * V + 1, dtype=dtype, device=DEV)[1:].view(B, R, V)
    gen2 = torch.Generator().manual_seed(V + 1)
    a = check_grad(x, tok, T, gen2, out=odd)
    gen2 = torch.Generator().manual_seed(V + 1)
    y = x.clone()
    g, h = torch.randn((B, R), generator=gen2), torch.randn((B, R), generator=gen2)
    saved = sv.spec_token_logprobs(y, tok.to(DEV), temperature=T)["saved"]
    b = sv.spec_token_logprobs_backward(y, tok.to(DEV), saved, g.to(DEV), h.to(DEV), temperature=T, out=y)
    assert b is y and torch.equal(a, b) and d.shape == x.shape


def test_gradient_against_differences():
    gen = torch.Generator().manual_seed(9)
    x = torch.randn((1, 2, 40), generator=gen).to(DEV)
    tok = torch.tensor([[3, 39]], dtype=torch.int32, device=DEV)
    f = lambda y: (lambda lp, e: (lp * torch.tensor([[1.0, -2.0]], device=DEV)).sum() + 0.5 * e.sum())(*sv.token_logprobs(y, tok, 0.9))  # noqa: E731
    y = x.clone().requires_grad_()
    f(y).backward()
    step = 2.0 ** -6      # differences of fp32 values: truncation ~ step^2, rounding ~ 2^-21 / step
    for r, j in ((0, 3), (0, 7), (1, 39), (1, 0), (1, 20)):
        e = torch.zeros_like(x)
        e[0, r, j] = step
        d = (f(x + e).double() - f(x - e).double()) / (2 * step)
        assert abs(float(d - y.grad[0, r, j])) < 4 * step ** 2 + 2.0 ** -20 / step


def test_graph_and_own_buffers():
    gen = torch.Generator().manual_seed(10)
    x = (torch.randn((2, 3, 9000), generator=gen) * 3).to(BF).to(DEV)
    tok = torch.randint(0, 9000, (2, 3), generator=gen, dtype=torch.int32).to(DEV)
    want = sv.spec_token_logprobs(x, tok, n_top=8)
    out = {k: torch.empty_like(v) for k, v in want.items()}
    ws = torch.full((sv.load_library().spec_token_logprobs_workspace_size(6, 9000, 1, 8),), 0xff, dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.spec_token_logprobs(x, tok, n_top=8, workspace=ws, out=out)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(out[k], want[k]), k


@pytest.mark.parametrize("of", ["logprob", "entropy", "product"])
def test_a_second_derivative_is_an_error(of):
    """Also where the upstream gradients are constants, as a sum's are: the gradient still depends on the logits."""
    x = torch.randn((1, 2, 40), generator=torch.Generator().manual_seed(11)).to(DEV).requires_grad_()
    tok = torch.tensor([[3, 39]], dtype=torch.int32, device=DEV)
    lp, ent = sv.token_logprobs(x, tok)
    loss = dict(logprob=lp, entropy=ent, product=lp * ent)[of].sum()
    first, = torch.autograd.grad(loss, x, retain_graph=True)
    again, = torch.autograd.grad(loss, x, create_graph=True)
    assert torch.equal(first, again) and not first.requires_grad
    with pytest.raises(sv.SpecVerifyError):
        (sv.token_logprobs(x, tok)[0].sum() + (again ** 2).sum()).backward()


def test_tokens_past_32_bits_are_out_of_range():
    x = torch.randn((1, 3, 50), generator=torch.Generator().manual_seed(12)).to(DEV)
    r = sv.spec_token_logprobs(x, torch.tensor([[2 ** 32 + 3, 3, -2 ** 32 + 3]], device=DEV))
    bad = sv.STATUS_BAD_TOKEN
    assert r["status"].tolist() == [[bad, 0, bad]] and r["logprob"][0, 0] == 0 and r["logprob"][0, 2] == 0


def test_tokens_of_the_differentiable_call_may_be_a_list():
    x = torch.randn((1, 2, 40), generator=torch.Generator().manual_seed(13)).to(DEV).requires_grad_()
    grads = []
    for tok in ([[3, -1]], torch.tensor([[3, -1]]), torch.tensor([[3, -1]], dtype=torch.int32, device=DEV)):
        lp, ent = sv.token_logprobs(x, tok)
        grads.append(torch.autograd.grad((lp + ent).sum(), x)[0])
    assert torch.equal(grads[0], grads[1]) and torch.equal(grads[0], grads[2])
