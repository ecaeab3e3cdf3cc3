"""Token log probabilities and their gradient on the GPU against float64 (logprob_ref)."""

import numpy as np
import pytest

import logprob_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    import torch
    import rejection_sampling_verify_10_amd as R
    assert torch.cuda.is_available(), "GPU test without a GPU"
    R.lib()
    return R


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def logits(rng, rows, V, dtype, pad=0, size=3.0):
    """Rows of a wider tensor (pad elements between them) and their values."""
    import torch
    z = size * rng.standard_normal((rows, V + pad)) - 1.1 * np.log(1 + rng.permutation(V + pad))
    t = dev(z.astype(np.float32))
    t = (t.bfloat16() if dtype == "bf16" else t)[:, :V]
    return t, t.float().cpu().numpy()


def check(r, want, top_n):
    lp, h = r.logprobs.cpu().numpy().reshape(len(want), -1), r.entropy.cpu().numpy().ravel()
    for i, w in enumerate(want):
        np.testing.assert_array_equal(np.isfinite(lp[i]), np.isfinite(w["lp"]), err_msg=f"row {i}")
        np.testing.assert_array_equal(np.isnan(lp[i]), np.isnan(w["lp"]))
        ok = np.isfinite(w["lp"])
        assert (np.abs(lp[i][ok] - w["lp"][ok]) <= w["lp_tol"][ok]).all(), (i, lp[i], w["lp"], w["lp_tol"])
        assert np.isnan(h[i]) == np.isnan(w["h"])
        if not np.isnan(w["h"]):
            assert abs(h[i] - w["h"]) <= w["h_tol"], (i, h[i], w["h"], w["h_tol"])
        if top_n:
            ids, tl = r.top_tokens.cpu().numpy().reshape(-1, top_n)[i], r.top_logprobs.cpu().numpy().reshape(-1, top_n)[i]
            np.testing.assert_array_equal(ids, w["top"], err_msg=f"row {i}")
            ok = np.isfinite(w["top_lp"])
            np.testing.assert_array_equal(np.isfinite(tl), ok)
            np.testing.assert_array_equal(np.isnan(tl), np.isnan(w["top_lp"]))
            assert (np.abs(tl[ok] - w["top_lp"][ok]) <= w["top_tol"][ok]).all()


def check_grad(got, want, tol):
    got = got.float().cpu().numpy().reshape(want.shape)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    off = np.abs(got - want)[ok] - tol[ok]
    assert (off <= 0).all(), off.max()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,V,M,top,T,pad", [
    (1, 1, 1, 1, 1.0, 0), (3, 2, 2, 64, 0.7, 0), (2, 7, 1, 5, 1.0, 0), (4, 9, 3, 64, 1.3, 3), (5, 255, 64, 20, 1.0, 0),
    (3, 4097, 1, 5, 0.7, 7), (700, 1001, 2, 3, 1.0, 0), (2, 32000, 8, 20, 1.0, 0), (9, 50257, 1, 1, 0.25, 0),
    (1, 128256, 1, 5, 1.0, 0), (520, 20011, 1, 64, 1.0, 5), (200, 128256, 1, 20, 0.7, 0), (1, 262147, 1, 0, 1.0, 0),
])
def test_forward_and_gradient(R, dtype, rows, V, M, top, T, pad):
    rng = np.random.default_rng([rows, V, M, top])
    z, zv = logits(rng, rows, V, dtype, pad)
    tokens = rng.integers(0, V, (rows, M)).astype(np.int32)
    tokens[rng.random((rows, M)) < 0.2] = -1                   # some tokens missing, some rows without any
    if rows > 2:
        tokens[1] = -1
    r = R.token_logprobs(z, dev(tokens), T, top)
    few = np.arange(rows) if rows * V < 3e6 else rng.choice(rows, 24, replace=False)
    want = ref.forward(zv[few], tokens[few], T, top)
    pick = lambda t: None if t is None else t[dev(few.astype(np.int64))]     # noqa: E731
    check(R.TokenLogprobs(*map(pick, r)), want, top)
    g = rng.standard_normal((rows, M)).astype(np.float32)
    gh = rng.standard_normal(rows).astype(np.float32)
    for entropy in (None, gh):
        got = R.token_logprobs_grad(z, dev(tokens), r.stats, dev(g), None if entropy is None else dev(entropy), T)
        assert got.dtype == z.dtype and got.shape == z.shape
        check_grad(pick(got), *ref.backward(zv[few], tokens[few], g[few], None if entropy is None else entropy[few], T, dtype))


def odd_rows(V, dtype):
    """Rows that an implementation may stumble over."""
    import torch
    rng = np.random.default_rng(5)
    low = torch.finfo(torch.bfloat16 if dtype == "bf16" else torch.float32).min
    base = rng.standard_normal((11, V)).astype(np.float32)
    base[0, 1:] = -np.inf                                     # one token left
    base[1, : V // 2] = -np.inf                               # half masked
    base[2, V // 2:] = low                                    # masked by the type's lowest value
    base[3] = low                                             # nothing but it
    base[4] = -np.inf                                         # nothing at all: NaN
    base[5, V - 1] = np.nan
    base[6, 3] = np.inf
    base[7] = 0.5                                             # ties everywhere
    base[8, ::3] = 7.0                                        # many ties at the top
    base[9] = 1e-30 * base[9]
    base[10] = 3e4 * base[10]
    z = dev(base)
    z = z.bfloat16() if dtype == "bf16" else z
    return z, z.float().cpu().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [64, 1003, 70001])
@pytest.mark.parametrize("T", [1.0, 0.01])
def test_odd_rows(R, dtype, V, T):
    z, zv = odd_rows(V, dtype)
    n = z.shape[0]
    tokens = np.stack([np.zeros(n), np.full(n, V - 1), np.full(n, 1)], 1).astype(np.int32)
    r = R.token_logprobs(z, dev(tokens), T, 20)
    want = ref.forward(zv, tokens, T, 20)
    # differences of the lowest value from a number next to it pass float32's range
    for w in want:
        for k in ("lp", "top_lp"):
            with np.errstate(over="ignore"):
                w[k] = np.where(np.isfinite(w[k]), w[k].astype(np.float32), w[k]).astype(np.float64)
    check(r, want, 20)
    g, gh = np.ones((n, 3), np.float32), np.full(n, 0.5, np.float32)
    check_grad(R.token_logprobs_grad(z, dev(tokens), r.stats, dev(g), dev(gh), T),
               *ref.backward(zv, tokens, g, gh, T, dtype))


def test_tokens_out_of_range_and_none(R):
    rng = np.random.default_rng(1)
    z, zv = logits(rng, 4, 1000, "f32")
    tokens = np.array([[5, 1000], [-1, -7], [-1, 999], [2 ** 31 - 1, 3]], np.int32)
    r = R.token_logprobs(z, dev(tokens), 1.0, 2)
    check(r, ref.forward(zv, tokens, 1.0, 2), 2)
    g = rng.standard_normal((4, 2)).astype(np.float32)
    check_grad(R.token_logprobs_grad(z, dev(tokens), r.stats, dev(g)), *ref.backward(zv, tokens, g, None, 1.0, "f32"))
    # no tokens: every row is read
    r = R.token_logprobs(z, None, 1.0, 3)
    assert r.logprobs.numel() == 0
    check(r, ref.forward(zv, np.zeros((4, 0), np.int32), 1.0, 3), 3)


def test_rows_without_tokens_are_not_read(R):
    import torch
    z = torch.full((2, 5000), float("nan"), device="cuda")
    z[0] = 1.0
    tokens = dev(np.array([3, -1], np.int32))
    r = R.token_logprobs(z, tokens, 1.0, 2)
    assert abs(r.logprobs[0].item() + np.log(5000)) < 1e-5 and r.logprobs[1].item() == 0 and r.entropy[1].item() == 0
    assert r.top_tokens.tolist() == [[0, 1], [-1, -1]]
    g = R.token_logprobs_grad(z, tokens, r.stats, torch.ones(2, device="cuda"))
    assert (g[1] == 0).all() and not torch.isnan(g).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_same_token_twice_and_in_place(R, dtype):
    rng = np.random.default_rng(2)
    z, zv = logits(rng, 6, 9001, dtype, pad=3)
    tokens = rng.integers(0, 9001, (6, 4)).astype(np.int32)
    tokens[:, 2] = tokens[:, 0]
    tokens[3] = 9000
    g, gh = rng.standard_normal((6, 4)).astype(np.float32), rng.standard_normal(6).astype(np.float32)
    r = R.token_logprobs(z, dev(tokens))
    want, tol = ref.backward(zv, tokens, g, gh, 1.0, dtype)
    first = R.token_logprobs_grad(z, dev(tokens), r.stats, dev(g), dev(gh))
    check_grad(first, want, tol)
    got = R.token_logprobs_grad(z, dev(tokens), r.stats, dev(g), dev(gh), out=z)
    assert got is z and (got == first).all()


def test_gradient_against_differences(R):
    """Central differences of the float64 forward along random directions: their error is the third derivative's, eps^2."""
    rng = np.random.default_rng(3)
    z, zv = logits(rng, 3, 301, "f32")
    tokens = rng.integers(0, 301, (3, 2)).astype(np.int32)
    g, gh = rng.standard_normal((3, 2)).astype(np.float32), rng.standard_normal(3).astype(np.float32)
    T = 0.8
    r = R.token_logprobs(z, dev(tokens), T)
    grad = R.token_logprobs_grad(z, dev(tokens), r.stats, dev(g), dev(gh), T).double().cpu().numpy()

    def loss(a):
        w = ref.forward(a, tokens, T, 0)
        return sum((g[i] * w[i]["lp"]).sum() + gh[i] * w[i]["h"] for i in range(3))

    for _ in range(5):
        d = rng.standard_normal(zv.shape)
        eps = 1e-5
        slope = (loss(zv + eps * d) - loss(zv - eps * d)) / (2 * eps)
        assert abs((grad * d).sum() - slope) < 1e-4 * (1 + np.abs(grad * d).sum())


def test_workspace_is_shared_and_left_zero(R):
    import torch
    rng = np.random.default_rng(4)
    sizes = [(1, 128256, 5), (3, 50000, 64), (2, 128256, 0), (40, 128256, 20)]
    need = max(R.token_logprobs_workspace_bytes(r, V, n, torch.float32) for r, V, n in sizes)
    ws = R.new_workspace(need, torch.device("cuda", 0))
    for rows, V, n in sizes + sizes[::-1]:
        z, zv = logits(rng, rows, V, "f32")
        tokens = rng.integers(0, V, (rows, 1)).astype(np.int32)
        few = slice(0, min(rows, 3))
        r = R.token_logprobs(z, dev(tokens), 1.0, n, workspace=ws)
        assert not ws.any()
        check(R.TokenLogprobs(*(None if t is None else t[few] for t in r)), ref.forward(zv[few], tokens[few], 1.0, n), n)


def test_captured_and_replayed(R):
    import torch
    rng = np.random.default_rng(6)
    z, _ = logits(rng, 8, 128256, "bf16")
    tokens = dev(rng.integers(0, 128256, (8, 1)).astype(np.int32))
    g = torch.ones(8, 1, device="cuda")
    ws = R.new_workspace(R.token_logprobs_workspace_bytes(8, 128256, 5), z.device)
    run = lambda: (lambda r: (*r, R.token_logprobs_grad(z, tokens, r.stats, g)))(R.token_logprobs(z, tokens, 1.0, 5, workspace=ws))  # noqa: E731
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        run()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for k in range(3):
        z.copy_(logits(rng, 8, 128256, "bf16")[0])
        eager = [t.clone() for t in run()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, eager):
            assert torch.equal(a, b)


def test_two_graphs_share_a_workspace(R):
    """Rows in slices, replayed in turns with eager calls of other sizes between."""
    import torch
    rng = np.random.default_rng(16)
    ws = R.new_workspace(R.token_logprobs_workspace_bytes(9, 60000, 20), torch.device("cuda", torch.cuda.current_device()))
    graphs = []
    for rows, V, top in ((3, 60000, 20), (9, 32001, 5)):
        z, tokens = logits(rng, rows, V, "f32")[0], dev(rng.integers(0, V, (rows, 2)).astype(np.int32))
        call = lambda z=z, tokens=tokens, top=top: R.token_logprobs(z, tokens, 0.9, top, workspace=ws)   # noqa: E731
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call()
        graphs.append((graph, out, z, call))
    for k in range(4):
        for graph, _, z, _ in graphs:
            z.copy_(logits(rng, *z.shape, "f32")[0])
            graph.replay()
        for _, out, _, call in graphs:
            for a, b in zip(out, call()):
                assert torch.equal(a, b)
    assert not ws.any()


def test_offsets_past_32_bits(R):
    """Rows of a tensor of more than 2^31 elements: what they give in a small one (as many workgroups a row)."""
    import torch
    rng = np.random.default_rng(17)
    V, many = 128256, 17001
    at = [0, 8000, 16744, many - 1]
    few, _ = logits(rng, 4, V, "bf16")
    tok = dev(rng.integers(0, V, (4, 2)).astype(np.int32))
    got = []
    for rows, places in ((300, [0, 1, 2, 299]), (many, at)):
        z = torch.empty(rows, V, dtype=torch.bfloat16, device="cuda")
        z[places] = few
        tokens = torch.full((rows, 2), -1, dtype=torch.int32, device="cuda")
        tokens[places] = tok
        r = R.token_logprobs(z, tokens, 1.1, 4)
        g = R.token_logprobs_grad(z, tokens, r.stats, torch.ones(rows, 2, device="cuda"), torch.ones(rows, device="cuda"), 1.1, out=z)
        got.append([t[places].clone() for t in (*r, g)])
        for place in set(range(0, rows, 500)) - set(places):
            assert not g[place].any()
        del z, g
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_emitted_tokens_of_a_verification(R):
    """The chain's verification and its answer's log probabilities, as a server asks for them."""
    import torch
    rng = np.random.default_rng(7)
    B, K, V = 5, 4, 32000
    z, zv = logits(rng, B * (K + 1), V, "bf16")
    z = z.view(B, K + 1, V)
    q = torch.softmax(z[:, :K].float() + 0.5 * torch.randn(B, K, V, device="cuda"), -1)
    x = torch.multinomial(q.view(-1, V), 1).view(B, K).to(torch.int32)
    tokens, alen = R.verify_chain(z, q, x, torch.rand(B, K + 1, device="cuda"), 1.0, 0)
    r = R.token_logprobs(z, tokens, 1.0, 3)
    assert r.logprobs.shape == (B, K + 1) and r.top_tokens.shape == (B, K + 1, 3)
    flat = tokens.cpu().numpy().reshape(-1, 1)
    want = ref.forward(zv, flat, 1.0, 3)
    check(r, want, 3)
    emitted = (torch.arange(K + 1, device="cuda") <= alen.view(-1, 1))
    assert torch.equal(emitted, tokens >= 0) and (r.logprobs[emitted] < 0).all() and (r.logprobs[~emitted] == 0).all()


def small(T):
    """A temperature as the call gets it."""
    return float(np.float32(T))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1003, 70001])
@pytest.mark.parametrize("T", [1e-6, 1e-7, 3e-9, 1e-10, 1e-20, 1e-30])
def test_small_temperatures(R, dtype, V, T):
    """The product of a logit and log2(e)/T has no binary places left, and rounds by more than a power of two."""
    rng = np.random.default_rng(int(V - np.log(T)))
    z, zv = logits(rng, 40, V, dtype, size=6.0)
    tokens = np.stack([zv.argmax(1), rng.integers(0, V, 40), np.argsort(zv, 1)[:, -2]], 1).astype(np.int32)
    r = R.token_logprobs(z, dev(tokens), small(T), 4)
    check(r, ref.forward(zv, tokens, small(T), 4), 4)
    g = rng.standard_normal((40, 3)).astype(np.float32)
    check_grad(R.token_logprobs_grad(z, dev(tokens), r.stats, dev(g), None, small(T)), *ref.backward(zv, tokens, g, None, small(T), dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1003, 70001])
@pytest.mark.parametrize("low", [-2e9, -1e10, -1e30])
def test_rows_far_below_zero(R, dtype, V, low):
    """Rows masked as a whole by a large negative number, alike or nearly so; some of a row; one token left."""
    rng = np.random.default_rng(3)
    base = 3 * rng.standard_normal((5, V)).astype(np.float32)
    base[0] = low
    base[1] = low * (1 + 2.0 ** -7 * rng.integers(0, 3, V))
    base[2, 1:] = low
    base[3, : V // 2] = low
    base[4, V // 3:] += low
    z = dev(base)
    z = z.bfloat16() if dtype == "bf16" else z
    zv = z.float().cpu().numpy()
    tokens = np.stack([np.zeros(5), np.full(5, V - 1), zv.argmax(1)], 1).astype(np.int32)
    r = R.token_logprobs(z, dev(tokens), 1.0, 5)
    check(r, ref.forward(zv, tokens, 1.0, 5), 5)
    g = np.ones((5, 3), np.float32)
    check_grad(R.token_logprobs_grad(z, dev(tokens), r.stats, dev(g)), *ref.backward(zv, tokens, g, None, 1.0, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,h", [(1e-9, 1.0), (1e-20, -1.0), (1e-30, 1.0), (1.0, 1e10), (1e-37, 0.0)])
def test_gradient_where_a_factor_is_infinite(R, dtype, T, h):
    """Tokens of probability 0 get no gradient, however large what multiplies it."""
    rng = np.random.default_rng(8)
    z, zv = logits(rng, 9, 5003, dtype)
    z[1, ::2] = float("-inf")
    z[2, 1:] = float("-inf")
    zv = z.float().cpu().numpy()
    tokens = np.stack([zv.argmax(1), rng.integers(0, 5003, 9), np.full(9, 4)], 1).astype(np.int32)
    r = R.token_logprobs(z, dev(tokens), small(T))
    g, gh = np.full((9, 3), 0.5, np.float32), np.full(9, h, np.float32)
    g[:, 1:] = 0.25 if T > 1e-36 else 3.0                     # the last: (1/T) sum g passes float32
    got = R.token_logprobs_grad(z, dev(tokens), r.stats, dev(g), dev(gh), small(T)).float().cpu().numpy()
    want, tol = ref.backward(zv, tokens, g, gh, small(T), dtype)
    # what is within float32: all but the given tokens' own and the likeliest of the last
    fits = np.abs(want) + tol < 1e38
    assert not np.isnan(got).any() and fits.sum() > 9 * 4990
    assert (np.abs(got - want) <= tol)[fits].all()


def peaked(rng, rows, V, dtype):
    """Rows of one confident token, 20 to 39 powers of two above the rest, where a wave meets it early, late or last of all."""
    z = rng.standard_normal((rows, V)).astype(np.float32)
    r = np.arange(rows)
    at = np.array([0, 5, V // 3, V // 2, V - 700, V - 2, V - 1])[r % 7]
    z[r, at] = 4 + np.array([20, 24, 27, 30, 39])[r % 5] * np.log(2)
    t = dev(z)
    t = t.bfloat16() if dtype == "bf16" else t
    return t, t.float().cpu().numpy().astype(np.float64), at


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,V", [(8, 20011), (300, 20011), (300, 128256)])
def test_confident_rows(R, dtype, rows, V):
    """The sum is 1 and a little. Behind the peak it goes through 15 additions of a group's half, one of the halves, 16 of groups at
    most, each off by half a step of float32 above 1, which is 2^-24, in either direction: four times the root of the sum of
    their squares (a third of 2^-48 each); and the peak's own exponential by a step and by its exponent's rounding, 2^-24."""
    rng = np.random.default_rng(rows + V)
    z, y, at = peaked(rng, rows, V, dtype)
    tol = 4 * np.sqrt(32 / 3) * 2.0 ** -24 + 2.0 ** -23 + 2.0 ** -24
    r = R.token_logprobs(z, dev(at.astype(np.int32)), 1.0, 1)
    x = y - y[np.arange(rows), at][:, None]
    e = np.exp(x)
    e[np.arange(rows), at] = 0.0
    rest = e.sum(1)
    lp, h = -np.log1p(rest), np.log1p(rest) - (e * x).sum(1) / (1 + rest)
    assert np.abs(r.logprobs.double().cpu().numpy() - lp).max() < tol
    assert (np.abs(r.entropy.double().cpu().numpy() - h) < tol + 8 * 2.0 ** -24 * h).all()
    assert np.array_equal(r.top_tokens[:, 0].cpu().numpy(), at) and (r.logprobs <= 0).all()


@pytest.mark.parametrize("rows", [1, 8, 300])
def test_sums_past_32_bits(R, rows):
    """A token that is all but certain, whichever way its row is cut up: exponents are whole numbers here (log2(e)/T rounds to 1), so
    that the sum, 1 + 20010 * 2^-40, is off only by what the peak's own thread had of the rest, 40 elements."""
    import torch
    V = 20011
    for at in (0, 9000, V - 1):
        z = torch.zeros(rows, V, device="cuda")
        z[:, at] = 40.0
        r = R.token_logprobs(z, dev(np.full(rows, at, np.int32)), float(np.float32(np.log2(np.e))))
        rest = (V - 1) * 2.0 ** -40
        lp, h = -rest, rest * (1 + 40 * np.log(2))
        assert (r.logprobs.double() / lp - 1).abs().max() < 41 / V and (r.entropy.double() / h - 1).abs().max() < 41 / V


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M", [None, 0, 1, 3])
def test_autograd(R, dtype, M):
    """The graph's gradient is the call's, bit for bit; tokens of the leading shape (None), of M a row, or none (0)."""
    import torch
    rng = np.random.default_rng(9)
    z = logits(rng, 12, 5003, dtype, pad=5)[0].view(3, 4, 5003)
    shape = (3, 4) if M is None else (3, 4, M)
    tokens = None if M == 0 else dev(rng.integers(-1, 5003, shape).astype(np.int32))
    g = None if M == 0 else dev(rng.standard_normal(shape).astype(np.float32))
    gh = dev(rng.standard_normal((3, 4)).astype(np.float32))
    plain = R.token_logprobs(z, tokens, 0.7, 3)
    assert not plain.logprobs.requires_grad
    z.requires_grad_()
    with torch.no_grad():
        assert not R.token_logprobs(z, tokens, 0.7).entropy.requires_grad
    r = R.token_logprobs(z, tokens, 0.7, 3)
    for a, b in zip(r, plain):
        assert torch.equal(a, b)
    assert r.logprobs.requires_grad and r.entropy.requires_grad
    assert not (r.stats.requires_grad or r.top_tokens.requires_grad or r.top_logprobs.requires_grad)
    ids = torch.zeros(3, 4, dtype=torch.int32, device="cuda") if M == 0 else tokens
    none = torch.zeros_like(ids, dtype=torch.float32)
    zd = z.detach()
    want = R.token_logprobs_grad(zd, ids, r.stats, none if M == 0 else g, gh, 0.7)
    loss = (gh * r.entropy).sum() + (0 if M == 0 else (g * r.logprobs).sum())
    got, = torch.autograd.grad(loss, z, retain_graph=True)
    assert got.dtype == z.dtype and torch.equal(got, want)
    got, = torch.autograd.grad(r.entropy.sum(), z, retain_graph=True)     # one of the two alone, a gradient that is expanded
    assert torch.equal(got, R.token_logprobs_grad(zd, ids, r.stats, none, torch.ones_like(gh), 0.7))
    if M != 0:
        got, = torch.autograd.grad(r.logprobs.sum(), z, retain_graph=True)
        assert torch.equal(got, R.token_logprobs_grad(zd, ids, r.stats, none + 1, None, 0.7))
    got, = torch.autograd.grad(loss, z, create_graph=True)                # its own gradient is refused
    with pytest.raises(RuntimeError, match="grad"):
        got.float().sum().backward()
    loss = R.token_logprobs(z, tokens, 0.7).entropy.sum()
    R.token_logprobs_grad(zd, ids, r.stats, none, gh, 0.7, out=zd)        # the logits' memory now holds something else
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_a_draft_models_step(R):
    """Targets' tokens under a linear head: gradients of its weights and inputs against float64 autograd."""
    import torch
    g = torch.Generator("cuda").manual_seed(3)
    x = torch.randn(2, 9, 64, generator=g, device="cuda", requires_grad=True)
    w = torch.randn(1003, 64, generator=g, device="cuda", requires_grad=True)
    ids = torch.randint(0, 1003, (2, 9, 4), generator=g, device="cuda", dtype=torch.int32)
    p = torch.rand(2, 9, 4, generator=g, device="cuda")
    r = R.token_logprobs(x @ w.T, ids, 1.3)
    (-(p * r.logprobs).sum() - 0.1 * r.entropy.sum()).backward()
    xd, wd = (t.detach().double().requires_grad_() for t in (x, w))
    lp = ((xd @ wd.T) / 1.3).log_softmax(-1)
    (-(p * lp.gather(-1, ids.long())).sum() + 0.1 * (lp.exp() * lp).sum()).backward()
    # sums of 18 and 1003 float32 products, whose terms' roundings do not all point one way
    for a, b in ((x.grad, xd.grad), (w.grad, wd.grad)):
        assert (a - b).abs().max() < 64 * 2.0 ** -24 * b.abs().max()


def test_a_training_step_captured(R):
    """Forward and backward captured and replayed on other logits, with eager steps between."""
    import torch
    rng = np.random.default_rng(10)
    x = logits(rng, 4, 40000, "bf16")[0].clone().requires_grad_()
    tokens = dev(rng.integers(0, 40000, (4, 2)).astype(np.int32))

    def step():
        r = R.token_logprobs(x, tokens, 0.9)
        return torch.autograd.grad(r.logprobs.sum() + 0.2 * r.entropy.sum(), x)[0]

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        with torch.no_grad():
            x.copy_(logits(rng, 4, 40000, "bf16")[0])
        eager = step()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,V", [(3, 4099), (6, 50000), (270, 2003)])
@pytest.mark.parametrize("T", [1e-12, 1e-3, 0.7, 1e6, 1e30])
def test_rows_that_move_the_reference(R, dtype, rows, V, T):
    """Rising, falling, masked in part by -inf and by large numbers, lifted and lowered as a whole, with blocks and peaks."""
    import torch
    rng = np.random.default_rng(V + rows)
    z = 5 * rng.standard_normal((rows, V))
    for r in range(rows):
        a, b = np.sort(rng.integers(0, V + 1, 2))
        how = r % 9 if rows > 9 else (2 * r + V) % 9
        if how < 2:
            z[r] = np.sort(z[r])[:: 1 - 2 * how]
        elif how < 4:
            z[r, a:b] = -np.inf if how == 2 else rng.choice([-1e4, -1e10, -1e30, -3.3e38])
        elif how == 4:
            z[r] += rng.choice([1e5, -1e9, 1e20, -1e30])
        elif how == 5:
            z[r, a:b] += rng.choice([50, 1e3, 1e6])
        elif how == 6:
            z[r, a:] += 1e4
        elif how == 7:
            z[r, rng.random(V) < 0.5] = -np.inf
    t = dev(z.astype(np.float32))
    t = t.bfloat16() if dtype == "bf16" else t
    zv = t.float().cpu().numpy()
    tokens = np.stack([zv.argmax(1), rng.integers(0, V, rows), np.full(rows, V - 1)], 1).astype(np.int32)
    r = R.token_logprobs(t, dev(tokens), small(T), 5)
    want = ref.forward(zv, tokens, small(T), 5)
    for w in want:                                            # differences past float32's range
        for k in ("lp", "top_lp"):
            with np.errstate(over="ignore"):
                w[k] = np.where(np.isfinite(w[k]), w[k].astype(np.float32), w[k]).astype(np.float64)
    check(r, want, 5)
    g, gh = rng.standard_normal((rows, 3)).astype(np.float32), rng.standard_normal(rows).astype(np.float32)
    got = R.token_logprobs_grad(t, dev(tokens), r.stats, dev(g), dev(gh), small(T))
    check_grad(got, *ref.backward(zv, tokens, g, gh, small(T), dtype))
