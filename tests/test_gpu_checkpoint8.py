"""8-bit activation checkpoints on the GPU against their definition in 64 bits.

Stored integers and scale bytes are compared for equality, and so are restored
values (a product with a power of two; float16 rounds it once). The weight
gradient's products are exact; each of its at most t additions (twice or three
times as many for a dY taken apart into two or three terms) is off by at most
2^-23 of the sum of magnitudes so far, and the result by one rounding."""
import numpy as np
import pytest
import torch

import plain8

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
TERMS = {torch.float32: 3, torch.bfloat16: 1, torch.float16: 2}
SMALLEST = {torch.float32: 2.0**-149, torch.bfloat16: 2.0**-133, torch.float16: 2.0**-24}


@pytest.fixture(scope="module")
def E():
    from entropy_constrained_unbiased_b200 import build, ecasq
    assert torch.cuda.is_available()
    build.build()
    ecasq.load()
    yield ecasq
    ecasq.check_stalled()


def _x(seed, n, k, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, k), generator=g) * torch.exp(torch.randn((n, 1), generator=g)) * scale
    return x.to(dtype).cuda()


def _f64(t):
    return t.detach().cpu().double().numpy()


def _same(E, X, seed):
    q, b = E.checkpoint8(X, seed)
    qr, br = plain8.checkpoint(_f64(X), seed if isinstance(seed, int) else int(seed))
    np.testing.assert_array_equal(b.cpu().numpy(), br)
    np.testing.assert_array_equal(q.cpu().numpy(), qr)
    want = plain8.values(qr, br)
    for dtype in TYPES:
        top = torch.finfo(dtype).max
        x = E.checkpoint8_restore(q, b, dtype)
        ref = torch.from_numpy(np.clip(want, -top, top) if dtype == torch.float16 else want).to(dtype)
        assert x.dtype == dtype
        np.testing.assert_array_equal(_f64(x), _f64(ref))
    return q, b


SHAPES = [(1, 1), (1, 31), (1, 32), (1, 33), (2, 100), (5, 777), (64, 64), (17, 4096), (3, 4100), (300, 40), (2, 20000)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("t,k", SHAPES)
def test_store_and_restore(E, t, k, dtype):
    _same(E, _x(t + k, t, k, dtype), 1234567890123 + t)


@pytest.mark.parametrize("dtype", TYPES)
def test_block_edges(E, dtype):
    """Largest magnitudes at, above and below 127 times a power of two, tiny and huge blocks, zeros."""
    rows = []
    for e in (-140, -127, -126, -120, -24, -14, 0, 9, 100, 121):
        for c in (127.0, 126.0, 128.0, 63.5, 1.0, 127.5):
            r = torch.linspace(-1, 1, 32).double() * c * 2.0**e
            rows.append(r)
    rows.append(torch.zeros(32).double())
    X = torch.stack(rows)
    X = X.clamp(-torch.finfo(dtype).max, torch.finfo(dtype).max).to(dtype).cuda()
    _same(E, X, 7)


@pytest.mark.parametrize("dtype", TYPES)
def test_blocks_without_finite_values(E, dtype):
    X = _x(3, 6, 100, dtype)
    X[0, 0], X[1, 40], X[2, 99], X[5, 64] = float("nan"), float("inf"), -float("inf"), float("nan")
    if dtype != torch.float16:
        X[3, 33] = 127.0 * 2.0**121
        X[4, 33] = torch.finfo(dtype).max
    q, b = _same(E, X, 11)
    assert int((b == 255).sum()) == (4 if dtype == torch.float16 else 5)


def test_strides_and_neighbours(E):
    wide = _x(2, 9, 140, torch.bfloat16)
    for lo, hi in [(0, 100), (3, 90), (8, 72)]:
        _same(E, wide[::2, lo:hi], 5)
    L = E.load()
    X = _x(3, 4, 21, torch.float32)
    q = torch.full((4, 64), 77, dtype=torch.int8, device="cuda")
    s = torch.full((4, 16), 78, dtype=torch.uint8, device="cuda")
    assert L.ecasq_checkpoint8(X.data_ptr(), 0, 4, 21, 21, 9, None, q.data_ptr(), 64, s.data_ptr(), 16, None) == 0
    torch.cuda.synchronize()
    assert torch.all(q[:, 32:] == 77) and torch.all(s[:, 1:] == 78) and torch.all(q[:, 21:32] == 0)
    np.testing.assert_array_equal(q[:, :21].cpu().numpy(), plain8.checkpoint(_f64(X), 9)[0])


def test_checkpoint_in_memory_that_ends_with_its_entries(E):
    """The last row's padding is neither read nor needed, by the restore or the gradient: other bytes there change
    nothing, and memory without them is taken."""
    t, k, ldq, lds = 7, 77, 96, 16
    q, b = E.checkpoint8(_x(1, t, k, torch.float32), 3)
    dY = _x(2, t, 40, torch.bfloat16)
    want = [E.checkpoint8_restore(q, b, dtype) for dtype in TYPES] + [E.checkpoint8_wgrad(dY, q, b)]
    for fill in (0x80, 0x7F, 0xFF):
        qs = torch.empty((t - 1) * ldq + k, dtype=torch.uint8, device="cuda").fill_(fill).view(torch.int8)
        bs = torch.empty((t - 1) * lds + 3, dtype=torch.uint8, device="cuda").fill_(fill)
        q2, b2 = qs.as_strided((t, k), (ldq, 1)), bs.as_strided((t, 3), (lds, 1))
        q2.copy_(q)
        b2.copy_(b)
        got = [E.checkpoint8_restore(q2, b2, dtype) for dtype in TYPES] + [E.checkpoint8_wgrad(dY, q2, b2)]
        assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_seed_in_device_memory(E):
    X = _x(4, 10, 100, torch.bfloat16)
    for value in (5, 2**62 + 12345, -3):
        word = torch.tensor([value], device="cuda")
        q, b = E.checkpoint8(X, word)
        qi, bi = E.checkpoint8(X, value)
        assert torch.equal(q, qi) and torch.equal(b, bi)
        np.testing.assert_array_equal(q.cpu().numpy(), plain8.checkpoint(_f64(X), value & (2**64 - 1))[0])


def test_rounding_is_unbiased(E):
    """Mean over 4000 seeds: within 5 standard errors of a rounding (at most s/2 each) and its 2^-17 s of bias."""
    X = _x(5, 8, 96, torch.float32)
    total = torch.zeros((8, 96), dtype=torch.float64, device="cuda")
    for seed in range(4000):
        q, b = E.checkpoint8(X, seed)
        total += E.checkpoint8_restore(q, b).double()
    s = torch.exp2(b.double() - 127).repeat_interleave(32, 1)
    assert torch.all((total / 4000 - X.double()).abs() <= s * (5 * 0.5 / 4000**0.5 + 2.0**-17))


def _gradient_tolerance(dy, x, ref, terms, out):
    n = dy.shape[0] * terms
    size = np.abs(dy).T @ np.abs(x)
    return n * 2.0**-23 * size * 1.01 + torch.finfo(out).eps / 2 * np.abs(ref) * 1.01 + SMALLEST[out]


def _check_gradient(E, dY, q, b, out=None):
    dW = E.checkpoint8_wgrad(dY, q, b, out)
    x, dy = plain8.values(q.cpu().numpy(), b.cpu().numpy()), _f64(dY)
    ref = dy.T @ x
    out = dY.dtype if out is None else out
    assert dW.dtype == out and dW.shape == ref.shape
    err, tol = np.abs(_f64(dW) - ref), _gradient_tolerance(dy, x, ref, TERMS[dY.dtype], out)
    assert np.all(err <= tol), (float((err / tol).max()), np.argwhere(err > tol)[:4].tolist())
    return dW, ref


GRADIENTS = [(1, 1, 1), (1, 64, 64), (2, 3, 33), (15, 128, 128), (64, 256, 256), (65, 100, 31), (100, 129, 300),
             (127, 8, 1000), (128, 1000, 64), (200, 257, 513), (1000, 130, 258), (777, 250, 1000), (3000, 64, 96),
             (4097, 136, 72), (9001, 24, 40)]


@pytest.mark.parametrize("t,o,k", GRADIENTS)
def test_weight_gradient(E, t, o, k):
    q, b = E.checkpoint8(_x(t + o, t, k, torch.float32), 3)
    for dtype in TYPES:
        dY = _x(t + k, t, o, dtype, 0.01)
        _check_gradient(E, dY, q, b)
        _check_gradient(E, dY, q, b, torch.float32)


@pytest.mark.parametrize("t,o,k", [(130, 2500, 2400), (300, 40, 20000), (70, 20000, 300), (1500, 2600, 2100)])
def test_weight_gradient_of_more_tiles_than_pairs(E, t, o, k):
    """Pairs of CTAs that take several tiles each, of one accumulator or several."""
    q, b = E.checkpoint8(_x(t + o, t, k, torch.float32), 3)
    for dtype in TYPES:
        _check_gradient(E, _x(t + k, t, o, dtype, 0.01), q, b)


def test_weight_gradient_float32_sums(E):
    """float32 results over a long sum stay within 2e-6 of the norm: the sums are not kept in fewer bits."""
    q, b = E.checkpoint8(_x(1, 8192, 256, torch.float32), 3)
    for dtype in TYPES:
        dW, ref = _check_gradient(E, _x(2, 8192, 384, dtype, 0.01), q, b, torch.float32)
        assert np.linalg.norm(_f64(dW) - ref) <= 2e-6 * np.linalg.norm(ref)


@pytest.mark.parametrize("dtype", TYPES)
def test_weight_gradient_same_sign(E, dtype):
    """All products positive: the running sum is as large as it can be, within the same bound."""
    q, b = E.checkpoint8(_x(1, 5000, 70, torch.float32).abs(), 3)
    dW, ref = _check_gradient(E, _x(2, 5000, 80, dtype).abs(), q, b, torch.float32)
    assert np.linalg.norm(_f64(dW) - ref) <= 2e-6 * np.linalg.norm(ref)


def test_weight_gradient_long_sums_are_not_cut(E):
    """131072 positive products per entry: the sums do not drift towards zero. With outputs spread evenly over a binade
    the results' own roundings cancel in the mean: what stays of it is 5 standard errors of 2^-8 / 3^(1/2) each and
    2^-16 at the binade's ends. An accumulator may lose 2^-23 for each of its 64 steps, and each of the 128 that are
    joined adds a rounding of at most 2^-24."""
    t, o, k = 131072, 1792, 1536  # 42 tiles: the tokens are not split
    g = torch.Generator("cuda").manual_seed(1)
    q, b = E.checkpoint8(torch.rand((t, k), generator=g, device="cuda").bfloat16(), 5)
    dY = (torch.rand((t, o), generator=g, device="cuda") * (1 + torch.arange(o, device="cuda") / o)).bfloat16()
    ref = torch.zeros((o, k), dtype=torch.float64, device="cuda")
    for r in range(0, t, 16384):
        ref += dY[r : r + 16384].double().T @ E.checkpoint8_restore(q[r : r + 16384], b[r : r + 16384]).double()
    drift = (E.checkpoint8_wgrad(dY, q, b).double() - ref).sum() / ref.sum()
    assert abs(float(drift)) <= 64 * 2.0**-23 + 128 * 2.0**-24 + 5 * 2.0**-8 / 3**0.5 / (o * k) ** 0.5 + 2.0**-16
    drift = (E.checkpoint8_wgrad(dY, q, b, torch.float32).double() - ref).sum() / ref.sum()
    assert abs(float(drift)) <= 16 * 2.0**-23 + 512 * 2.0**-24


def test_weight_gradient_no_tokens(E):
    q, b = E.checkpoint8(torch.empty((0, 70), device="cuda"), 1)
    dW = E.checkpoint8_wgrad(torch.empty((0, 50), device="cuda"), q, b)
    assert dW.shape == (50, 70) and not dW.any()


def test_weight_gradient_strides(E):
    q, b = E.checkpoint8(_x(1, 400, 520, torch.float32), 3)
    wide = _x(2, 800, 300, torch.bfloat16)
    for dY in (wide[::2, :256], wide[:400, 8:209], wide[:400, 3:131], wide[400:, 1:2]):
        _check_gradient(E, dY, q, b)
    _check_gradient(E, wide[:100, :64], q[100:200], b[100:200])
    for dtype in (torch.float32, torch.float16):
        _check_gradient(E, wide.to(dtype)[::2, 5:77], q, b)


@pytest.mark.parametrize("dtype", TYPES)
def test_weight_gradient_huge_and_tiny_gradients(E, dtype):
    """The largest, the smallest normal and exact values of dY's type come through."""
    top, low = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
    X = torch.zeros((3, 40), device="cuda")
    X[0, 3], X[1, 5], X[2, 7] = 1.0, 1.0, 1.0
    q, b = E.checkpoint8(X, 1)
    dY = torch.zeros((3, 20), dtype=dtype, device="cuda")
    dY[0, 1], dY[1, 2], dY[2, 4] = top, -low, 1 + torch.finfo(dtype).eps
    dW = E.checkpoint8_wgrad(dY, q, b)
    assert dW[1, 3] == top and dW[2, 5] == -low and dW[4, 7] == dY[2, 4] and int((dW != 0).sum()) == 3


@pytest.mark.parametrize("dtype", TYPES)
def test_weight_gradient_of_small_entries(E, dtype):
    """Entries down to the type's smallest, brought back by a large X: exact products, except for the bits of float32
    entries that lie under 2^-133. One product per sum, so that nothing else is rounded but the result. (The largest float16
    entries are infinities, and so are their products.)"""
    q, b = E.checkpoint8(torch.full((1, 32), 2.0**100, device="cuda"), 1)
    low = torch.tensor([SMALLEST[dtype]], dtype=torch.float64).log2().int().item()
    m = 1 + torch.rand(64, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    dY = torch.cat([m * 2.0**e for e in range(low, low + 60)]).to(dtype).cuda()[None]
    dW = E.checkpoint8_wgrad(dY, q, b, torch.float32)
    want = dY[0].double() * 2.0**100
    cut = 2.0**-133 if dtype == torch.float32 else 0.0
    off = torch.where(want.isinf()[:, None] & (dW == want[:, None]), 0.0, (dW.double() - want[:, None]).abs())
    assert torch.all(off <= cut * 2.0**100)
    exact = dY[0].abs().double() >= (2.0**-110 if dtype == torch.float32 else 0.0)
    assert int(exact.sum()) >= 64 * 20 and torch.equal(dW[exact].double(), want[exact, None].expand(-1, 32))


def test_weight_gradient_not_finite(E):
    """NaN and infinities of dY reach their row of dW alone, a marked block of X its 32 columns alone."""
    X = _x(1, 150, 200, torch.float32)
    X[77, 70] = float("inf")
    q, b = E.checkpoint8(X, 3)
    for dtype in TYPES:
        dY = _x(2, 150, 90, dtype)
        dY[3, 5], dY[149, 60] = float("nan"), float("inf")
        dW = E.checkpoint8_wgrad(dY, q, b)
        bad = torch.zeros((90, 200), dtype=torch.bool, device="cuda")
        bad[:, 64:96] = True
        bad[5] = True
        assert torch.isnan(dW[bad]).all()
        rest = torch.ones(90, dtype=torch.bool, device="cuda")
        rest[5], rest[60] = False, False
        assert torch.isfinite(dW[rest][:, :64]).all() and torch.isfinite(dW[rest][:, 96:]).all()
        assert not torch.isfinite(dW[60]).any()


def test_overlapping_calls_and_repeats(E):
    """Calls on several streams at once give what they give alone, bit for bit."""
    work = []
    for i, (t, o, k) in enumerate([(3000, 64, 96), (500, 300, 200), (9001, 24, 40), (64, 256, 256)]):
        q, b = E.checkpoint8(_x(i, t, k, torch.bfloat16), i)
        work.append((_x(i + 9, t, o, TYPES[i % 3]), q, b))
    want = [E.checkpoint8_wgrad(*w) for w in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(5):
        got = []
        for s, w in zip(streams, work):
            with torch.cuda.stream(s):
                got.append(E.checkpoint8_wgrad(*w))
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_graph_replays_draw_new_bits(E):
    """A captured store and gradient, replayed with another seed word and other inputs, equal the eager calls."""
    X, dY = _x(1, 600, 100, torch.bfloat16), _x(2, 600, 64, torch.float16)
    word = torch.tensor([5], device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q, b = E.checkpoint8(X, word)
        dW = E.checkpoint8_wgrad(dY, q, b)
    other = torch.cuda.CUDAGraph()
    with torch.cuda.graph(other):
        dW2 = E.checkpoint8_wgrad(dY, q, b, torch.float32)
    for seed in (5, 6, 7):
        word.fill_(seed)
        X.copy_(_x(seed, 600, 100, torch.bfloat16))
        g.replay()
        other.replay()
        torch.cuda.synchronize()
        qe, be = E.checkpoint8(X, seed)
        assert torch.equal(q, qe) and torch.equal(b, be)
        assert torch.equal(dW, E.checkpoint8_wgrad(dY, qe, be))
        assert torch.equal(dW2, E.checkpoint8_wgrad(dY, qe, be, torch.float32))


# -- checkpoint_linear -----------------------------------------------------------------


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape,o", [((48, 64), 40), ((2, 5, 33), 7), ((64,), 8), ((3, 0, 32), 8)])
def test_linear_gradients(E, dtype, shape, o):
    """Forward, input and bias gradients are F.linear's; the weight gradient is the formula's with the stored values."""
    from entropy_constrained_unbiased_b200.linear import checkpoint_linear
    import torch.nn.functional as F
    g = torch.Generator().manual_seed(3)
    x = torch.randn(shape, generator=g).to(dtype).cuda().requires_grad_()
    w = torch.randn((o, shape[-1]), generator=g).to(dtype).cuda().requires_grad_()
    bias = torch.randn(o, generator=g).to(dtype).cuda().requires_grad_()
    y = checkpoint_linear(x, w, bias, seed=21)
    dy = torch.randn(y.shape, generator=g).to(dtype).cuda()
    assert torch.equal(y, F.linear(x, w, bias))
    dx, dw, db = torch.autograd.grad(y, (x, w, bias), dy)
    d2, x2 = dy.reshape(-1, o), x.detach().reshape(-1, shape[-1])
    want_dx = (d2.double() @ w.double()).reshape(x.shape)
    size = (d2.double().abs() @ w.double().abs()).reshape(x.shape)
    half = torch.finfo(dtype).eps / 2
    assert torch.all((dx.double() - want_dx).abs() <= half * want_dx.abs() * 1.01 + o * 2.0**-23 * size + SMALLEST[dtype])
    q, b = E.checkpoint8(x2, 21)
    assert torch.equal(dw, E.checkpoint8_wgrad(d2, q, b, dtype))
    want_db, n = d2.double().sum(0), max(1, d2.shape[0])
    assert torch.all((db.double() - want_db).abs()
                     <= half * want_db.abs() * 1.01 + n * 2.0**-24 * d2.double().abs().sum(0) + SMALLEST[dtype])


def test_linear_weight_gradient_by_differences(E):
    """With the stored values in x's place the layer is linear in w, so a central difference of the loss along a
    direction equals <dW, direction> up to the roundings of float64 and of the float32 gradient."""
    from entropy_constrained_unbiased_b200.linear import checkpoint_linear
    x, w = _x(1, 60, 70, torch.float32), _x(2, 50, 70, torch.float32).requires_grad_()
    y = checkpoint_linear(x, w, seed=4)
    c = _x(3, 60, 50, torch.float32)
    (y * c).sum().backward()
    q, b = E.checkpoint8(x, 4)
    xs = E.checkpoint8_restore(q, b).double()
    direction = _x(5, 50, 70, torch.float32).double()
    loss = lambda m: (xs @ m.T * c.double()).sum()
    h = 1e-3
    slope = (loss(w.double() + h * direction) - loss(w.double() - h * direction)) / (2 * h)
    size = (c.double().abs().T @ xs.abs() * direction.abs()).sum()
    assert (slope - (w.grad.double() * direction).sum()).abs() <= 3 * 60 * 2.0**-23 * size


@pytest.mark.parametrize("k", [512, 768, 777])
def test_linear_under_saved_tensor_hooks(E, k):
    """What the layer keeps may be copied elsewhere and back (offload), whatever the width."""
    from entropy_constrained_unbiased_b200.linear import checkpoint_linear
    x, w = _x(1, 20, k, torch.bfloat16), _x(2, 10, k, torch.bfloat16).requires_grad_()
    dy = _x(3, 20, 10, torch.bfloat16)
    (want,) = torch.autograd.grad(checkpoint_linear(x, w, seed=3), w, dy)
    with torch.autograd.graph.save_on_cpu():
        y = checkpoint_linear(x, w, seed=3)
    assert torch.equal(torch.autograd.grad(y, w, dy)[0], want)
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t.clone(memory_format=torch.contiguous_format), lambda t: t):
        y = checkpoint_linear(x[:1], w, seed=3)
        z = checkpoint_linear(x[:0], w, seed=3)
    (got,) = torch.autograd.grad(y, w, dy[:1])
    assert torch.equal(got, torch.autograd.grad(checkpoint_linear(x[:1], w, seed=3), w, dy[:1])[0])
    assert not torch.autograd.grad(z, w, dy[:0])[0].any()


def test_linear_mean_gradient(E):
    """The mean over seeds is the gradient of the unrounded layer, within 5 standard errors."""
    from entropy_constrained_unbiased_b200.linear import checkpoint_linear
    x, w = _x(1, 20, 64, torch.float32), _x(2, 10, 64, torch.float32).requires_grad_()
    dy = _x(3, 20, 10, torch.float32)
    n, total = 2000, 0
    for seed in range(n):
        total = total + torch.autograd.grad(checkpoint_linear(x, w, seed=seed), w, dy)[0].double()
    _, b = E.checkpoint8(x, 0)
    s = torch.exp2(b.double() - 127).repeat_interleave(32, 1)
    spread = torch.sqrt((dy.double() ** 2).T @ (s / 2) ** 2)  # at most, for one seed
    bias = dy.double().abs().T @ s * 2.0**-17
    assert torch.all((total / n - dy.double().T @ x.double()).abs() <= 5 * spread / n**0.5 + bias + 1e-6)


def test_linear_of_a_sum_and_without_weight_gradient(E):
    from entropy_constrained_unbiased_b200.linear import checkpoint_linear
    x, w = _x(1, 20, 64, torch.bfloat16).requires_grad_(), _x(2, 10, 64, torch.bfloat16).requires_grad_()
    checkpoint_linear(x, w, seed=1).sum().backward()  # an expanded gradient
    q, b = E.checkpoint8(x.detach(), 1)
    assert torch.equal(w.grad, E.checkpoint8_wgrad(torch.ones((20, 10), dtype=torch.bfloat16, device="cuda"), q, b))
    y = checkpoint_linear(x, w.detach(), seed=1)
    x.grad = None
    y.sum().backward()
    assert x.grad is not None
    with torch.no_grad():
        assert not checkpoint_linear(x, w, seed=1).requires_grad


def test_linear_without_gradients_stores_nothing(E):
    """Evaluation with trainable weights is F.linear: no kernel of the library runs."""
    from entropy_constrained_unbiased_b200.linear import checkpoint_linear
    import torch.nn.functional as F
    x, w = _x(1, 20, 64, torch.bfloat16), _x(2, 10, 64, torch.bfloat16).requires_grad_()
    L = E.load()
    before = L.ecasq_launch_count(0)
    for mode in (torch.no_grad, torch.inference_mode):
        with mode():
            assert torch.equal(checkpoint_linear(x, w, seed=1), F.linear(x, w))
    assert L.ecasq_launch_count(0) == before
    checkpoint_linear(x, w, seed=1)
    assert L.ecasq_launch_count(0) == before + 1


def test_linear_refusals(E):
    """Layers without inputs or outputs are refused in the forward call, not by the backward pass; second derivatives
    and transforms by torch."""
    from entropy_constrained_unbiased_b200.linear import checkpoint_linear
    x, w = _x(1, 4, 8, torch.float32), _x(2, 6, 8, torch.float32).requires_grad_()
    for a, b in ((x, w[:0]), (x[:, :0], w[:, :0]), (x, w[:, :4]), (x, w[0])):
        with pytest.raises(E.EcasqError):
            checkpoint_linear(a, b, seed=1)
    y = checkpoint_linear(x.requires_grad_(), w, seed=1)
    (dw,) = torch.autograd.grad(y.square().sum(), w, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(dw.sum(), w)
    with pytest.raises(RuntimeError):
        torch.func.grad(lambda m: checkpoint_linear(x.detach(), m, seed=1).sum())(w.detach())


def test_linear_under_autocast(E):
    from entropy_constrained_unbiased_b200.linear import checkpoint_linear
    x, w = _x(1, 20, 64, torch.float32).requires_grad_(), _x(2, 10, 64, torch.float32).requires_grad_()
    with torch.autocast("cuda", dtype=torch.bfloat16):
        y = checkpoint_linear(x, w, seed=1)
    assert y.dtype == torch.bfloat16
    y.float().square().sum().backward()
    assert w.grad.dtype == torch.float32 and x.grad.dtype == torch.float32


def test_training_and_serving_together(E):
    """Two layers trained for a few steps with 8-bit checkpoints, then served from 8-bit weights: every gradient is
    finite, the checkpoint is what the backward pass reads, and the served outputs are near the trained ones."""
    from entropy_constrained_unbiased_b200.linear import checkpoint_linear, int8_linear
    torch.manual_seed(0)
    w1 = (torch.randn(96, 64, device="cuda") / 8).requires_grad_()
    w2 = (torch.randn(32, 96, device="cuda") / 10).requires_grad_()
    x = torch.randn(128, 64, device="cuda")
    target = torch.randn(128, 32, device="cuda")
    for step in range(3):
        h = torch.relu(checkpoint_linear(x, w1, seed=2 * step))
        loss = (checkpoint_linear(h, w2, seed=2 * step + 1) - target).square().mean()
        g1, g2 = torch.autograd.grad(loss, (w1, w2))
        assert torch.isfinite(g1).all() and torch.isfinite(g2).all() and g1.any() and g2.any()
        with torch.no_grad():
            w1 -= 0.1 * g1
            w2 -= 0.1 * g2
    with torch.no_grad():
        (q1, s1, _), (q2, s2, _) = E.int8_quantize(w1.detach()), E.int8_quantize(w2.detach())
        y = torch.relu(x @ w1.T) @ w2.T
        y8 = int8_linear(torch.relu(int8_linear(x, q1, s1)), q2, s2)
    assert (y8 - y).norm() <= 0.05 * y.norm()


def test_linear_of_transposed_and_expanded_inputs(E):
    from entropy_constrained_unbiased_b200.linear import checkpoint_linear, int8_linear
    base = _x(1, 64, 20, torch.float32)
    w = _x(2, 10, 64, torch.float32).requires_grad_()
    wq, ws, _ = E.int8_quantize(w.detach())
    for x in (base.T, base[:, :1].T.expand(20, 64), base.T.reshape(4, 5, 64).transpose(0, 1)):
        y = checkpoint_linear(x, w, seed=1)
        c = _x(3, y.numel(), 1, torch.float32).reshape(y.shape)
        (dw,) = torch.autograd.grad(y, w, c)
        q, b = E.checkpoint8(x.reshape(-1, 64).contiguous(), 1)
        assert torch.equal(dw, E.checkpoint8_wgrad(c.reshape(-1, 10), q, b))
        assert torch.equal(int8_linear(x, wq, ws), int8_linear(x.contiguous(), wq, ws))


def test_chained_launches_read_what_the_kernel_before_wrote(E):
    """Calls of two and three kernels back to back on one stream, whose workspaces the allocator gives to each in turn:
    each result is that of its own inputs (token scales, quantised tokens, bf16 terms, partial sums)."""
    wq, ws, _ = E.int8_quantize(_x(1, 300, 4096, torch.float32))
    xs = [[_x(100 * m + i, m, 4096, torch.bfloat16, 2.0**i) for i in range(4)] for m in (2, 9, 100, 300)]
    q, b = E.checkpoint8(_x(2, 6000, 96, torch.float32), 3)
    dys = [_x(50 + i, 6000, 64, dtype, 2.0**i) for dtype in TYPES for i in range(3)]
    def separately(x):
        a, s, _ = E.int8_quantize(x)
        torch.cuda.synchronize()
        return E.int8_matmul(a, s, wq, ws, None, x.dtype)
    want = [[separately(x) for x in group] for group in xs]
    for _ in range(20):
        for group, w in zip(xs, want):
            got = [E.int8_linear(x, wq, ws) for x in group]
            assert all(torch.equal(g, r) for g, r in zip(got, w))
        grads = [E.checkpoint8_wgrad(dY, q, b) for dY in dys]
        torch.cuda.synchronize()
        for dY, dW in zip(dys, grads):
            assert torch.equal(dW, E.checkpoint8_wgrad(dY, q, b))
    for dY, dW in zip(dys, grads):
        _check_gradient(E, dY, q, b)


def test_training_step_in_a_graph(E):
    """Forward and backward captured once and replayed with new inputs and a new seed word equal the eager step."""
    from entropy_constrained_unbiased_b200.linear import checkpoint_linear
    x, w = _x(1, 96, 64, torch.bfloat16), _x(2, 40, 64, torch.bfloat16).requires_grad_()
    c, word = _x(3, 96, 40, torch.bfloat16), torch.tensor([9], device="cuda")
    step = lambda seed: torch.autograd.grad(checkpoint_linear(x, w, seed=seed), w, c)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(word)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dw = step(word)
    for seed in (9, 10):
        word.fill_(seed)
        x.copy_(_x(seed, 96, 64, torch.bfloat16))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(dw, step(seed))


def test_offsets_past_32_bits(E):
    """More than 2^31 entries: the last rows of every operator equal those of the rows alone (the checkpoint's
    random bits go by the row's number, so its rows are compared with the definition)."""
    t, k = 70001, 32768
    X = torch.empty((t, k), dtype=torch.bfloat16, device="cuda")
    X.normal_(generator=torch.Generator("cuda").manual_seed(1))
    q, b = E.checkpoint8(X, 5)
    x = E.checkpoint8_restore(q, b, torch.bfloat16)
    want = plain8.checkpoint(_f64(X[-2:]), 5, t - 2)
    np.testing.assert_array_equal(q[-2:].cpu().numpy(), want[0])
    np.testing.assert_array_equal(b[-2:].cpu().numpy(), want[1])
    np.testing.assert_array_equal(_f64(x[-2:]), plain8.values(*want))
    dY = torch.zeros((t, 8), dtype=torch.bfloat16, device="cuda")
    dY[-2:] = _x(2, 2, 8, torch.bfloat16)
    dW = E.checkpoint8_wgrad(dY, q, b, torch.float32)
    ref = _f64(dY[-2:]).T @ plain8.values(*want)
    assert np.all(np.abs(_f64(dW) - ref) <= 2.0**-22 * (np.abs(_f64(dY[-2:])).T @ np.abs(plain8.values(*want))) + 1e-30)
    del x, q, b, dY, dW
    a, s, _ = E.int8_quantize(X)
    last, ls, _ = E.int8_quantize(X[-3:].clone())
    assert torch.equal(a[-3:], last) and torch.equal(s[-3:], ls)
    B, sb, _ = E.int8_quantize(_x(3, 24, k, torch.float32))
    assert torch.equal(E.int8_matmul(a, s, B, sb)[-3:], E.int8_matmul(last, ls, B, sb))
    assert torch.equal(E.int8_matmul(B, sb, a, s)[:, -3:], E.int8_matmul(B, sb, last, ls))
