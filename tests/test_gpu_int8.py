"""The integer linear layer on the GPU against its definition in 64 bits.

The quantiser is compared for equality (the integers follow from the exact
quotient, the scale is one float32 division). The product's integer sum is
exact, so an output may be off by four float32 roundings (the conversion of the
sum, two scales, the bias) of at most 2^-24 each, and one of the output type."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import plain8

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
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


def _same_rows(E, X):
    q, s, st = E.int8_quantize(X)
    qr, sr, bad = plain8.int8_rows(_f64(X))
    np.testing.assert_array_equal(q.cpu().numpy(), qr)
    np.testing.assert_array_equal(s.cpu().numpy(), sr)
    np.testing.assert_array_equal(st.cpu().numpy(), np.where(bad, E.ERR_RANGE, 0))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,k", [(1, 1), (1, 4096), (3, 7), (5, 32), (200, 33), (300, 1000), (149, 1025), (2, 4097),
                                 (3, 16384), (2, 40001), (1, 131072)])
def test_quantizer(E, n, k, dtype):
    _same_rows(E, _x(n * 7 + k, n, k, dtype))


@pytest.mark.parametrize("dtype", TYPES)
def test_quantizer_ties_and_sizes(E, dtype):
    """Every tie of a row (x / a = (j + 1/2) / 127 with a = 127 2^e), zeros, the smallest and largest values."""
    j = torch.arange(-127, 128).double()
    rows = [torch.cat([torch.tensor([127.0]), j / 2]) * 2.0**e for e in (-10, 0, 3)]
    big, tiny = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
    rows += [torch.zeros(256), torch.linspace(-1, 1, 256).double() * big, torch.linspace(-1, 1, 256).double() * tiny,
             torch.cat([torch.zeros(255), torch.tensor([SMALLEST[dtype]])])]
    _same_rows(E, torch.stack([r.double() for r in rows]).to(dtype).cuda())


@pytest.mark.parametrize("dtype", TYPES)
def test_quantizer_rows_without_a_scale(E, dtype):
    X = _x(1, 6, 300, dtype)
    X[1, 299] = float("nan")
    X[3, 0] = float("inf")
    X[4, 7] = -float("inf")
    X[5] = 0
    _same_rows(E, X)


def test_quantizer_strides_and_neighbours(E):
    """Rows inside a wider matrix, starting off the 16-byte boundary; the bytes around q stay as they were."""
    wide = _x(2, 9, 140, torch.bfloat16)
    for lo, hi in [(0, 100), (3, 90), (8, 72)]:
        _same_rows(E, wide[::2, lo:hi])
    L = E.load()
    X = _x(3, 4, 21, torch.float32)
    q = torch.full((4, 32), 77, dtype=torch.int8, device="cuda")
    s, st = torch.empty(4, device="cuda"), torch.empty(4, dtype=torch.int32, device="cuda")
    assert L.ecasq_int8_quantize(X.data_ptr(), 0, 4, 21, 21, q.data_ptr(), 32, s.data_ptr(), st.data_ptr(), None) == 0
    torch.cuda.synchronize()
    assert torch.all(q[:, 21:] == 77)
    np.testing.assert_array_equal(q[:, :21].cpu().numpy(), plain8.int8_rows(_f64(X))[0])


def _operands(seed, m, n, k, full=False):
    g = torch.Generator().manual_seed(seed)
    def rows(r):
        t = torch.zeros((r, (k + 31) // 32 * 32), dtype=torch.int8)
        t[:, :k] = 127 if full else torch.randint(-127, 128, (r, k), generator=g, dtype=torch.int8)
        return t.cuda()[:, :k]
    A, B = rows(m), rows(n)
    sa, sb = torch.rand(m, generator=g).cuda() + 0.01, torch.rand(n, generator=g).cuda() * 1e-3
    return A, sa, B, sb, torch.randn(n, generator=g).cuda()


def _check_product(E, A, sa, B, sb, bias, dtype):
    Y = E.int8_matmul(A, sa, B, sb, bias, dtype)
    acc = (A.double() @ B.double().T).cpu().numpy()  # integers below 2^53: exact
    p = acc * _f64(sa)[:, None] * _f64(sb)
    ref = p if bias is None else p + _f64(bias)
    size = np.abs(p) + (0 if bias is None else np.abs(_f64(bias)))
    tol = 4 * 2.0**-24 * size * 1.01 + torch.finfo(dtype).eps / 2 * np.abs(ref) * 1.01 + SMALLEST[dtype]
    assert Y.shape == (A.shape[0], B.shape[0]) and Y.dtype == dtype
    err = np.abs(_f64(Y) - ref)
    assert np.all(err <= tol), (float((err / tol).max()), np.argwhere(err > tol)[:4].tolist())


SHAPES = [(1, 1, 1), (1, 64, 4096), (1, 4099, 4096), (2, 3001, 33), (3, 5, 16), (4, 130, 515), (8, 1000, 1024),
          (9, 257, 640), (16, 4096, 4096), (17, 129, 100), (31, 64, 2048), (33, 300, 129), (64, 16384, 128),
          (65, 65, 65), (100, 1000, 4099), (128, 128, 128), (129, 513, 257), (256, 256, 4096), (300, 700, 1000),
          (511, 255, 127), (1000, 300, 3001), (2049, 1025, 384), (4096, 512, 64)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(E, m, n, k):
    A, sa, B, sb, bias = _operands(m + n + k, m, n, k)
    for i, dtype in enumerate(TYPES):
        _check_product(E, A, sa, B, sb, bias if i != 1 else None, dtype)


@pytest.mark.parametrize("m,n,k", [(1300, 4400, 640), (4500, 4200, 200), (20000, 300, 100), (300, 20000, 96)])
def test_product_of_more_tiles_than_pairs(E, m, n, k):
    """Pairs of CTAs that take several tiles each (either accumulator and its token scales in turn), channels beyond the
    first block of 4096."""
    A, sa, B, sb, bias = _operands(m + n + k, m, n, k)
    for i, dtype in enumerate(TYPES):
        _check_product(E, A, sa, B, sb, bias if i != 1 else None, dtype)


@pytest.mark.parametrize("m", [1, 20, 300])
def test_product_largest_sums(E, m):
    """Every product 127^2 at the longest sum: just below 2^31."""
    A, sa, B, sb, _ = _operands(5, m, 40, 131072, full=True)
    _check_product(E, A, sa, B, sb, None, torch.float32)


@pytest.mark.parametrize("m", [1, 2, 20, 300])
def test_product_of_the_least_integers(E, m):
    """Every product (-128)^2 at the longest sum is 2^31; its neighbours, and the least sum, lie inside 32 bits."""
    A = torch.full((m, 131072), -128, dtype=torch.int8, device="cuda")
    B = torch.full((140, 131072), -128, dtype=torch.int8, device="cuda")
    B[1, 5], B[2, 7], B[3] = -127, 127, 127
    ones = torch.ones(300, device="cuda")
    Y = E.int8_matmul(A, ones[:m], B, ones[:140], None, torch.float32)
    want = torch.full((140,), 2**31, dtype=torch.float64, device="cuda")
    want[1], want[2], want[3] = 2**31 - 128, 2**31 - 128 * 255, -128 * 127 * 131072
    assert torch.equal(Y, want.float().expand(m, 140))


@pytest.mark.parametrize("m", [2, 20, 300])
@pytest.mark.parametrize("ea,eb", [(118, -60), (96, 0), (-133, 100), (-140, 110), (-94, 0), (60, 40), (-100, -20), (100, 100)])
def test_product_with_extreme_scales(E, m, ea, eb):
    """Token scales near either end of float32: what the two scales give together is what counts."""
    A, sa, B, sb, bias = _operands(3, m, 40, 4096)
    sa, sb = (sa.double() * 2.0**ea).float(), (sb.double() * 2.0**eb).float()
    sa[0], A[0, 7] = 0, 5
    if ea + eb == 200:
        Y = E.int8_matmul(A, sa, B, sb, bias, torch.float32)
        assert torch.equal(Y[0], bias) and torch.isinf(Y[1:]).all()
        return
    _check_product(E, A, sa, B, sb, None, torch.float32)
    _check_product(E, A, sa, B, sb, bias, torch.float32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m", [1, 12, 200])
def test_linear_of_huge_and_tiny_tokens(E, m, dtype):
    """Tokens near the type's largest values, and near its smallest, through weights that bring them back."""
    w = torch.randn((30, 512), generator=torch.Generator().manual_seed(1)).cuda()
    x = torch.randn((m, 512), generator=torch.Generator().manual_seed(2)).clamp(-3, 3).cuda()
    for ex, ew in ((126, -30), (-126, 90)):
        wq, ws, _ = E.int8_quantize(w * 2.0**ew)
        t = (x.double() * 2.0**ex / 4).to(dtype)
        q, s, _ = E.int8_quantize(t)
        y = E.int8_linear(t, wq, ws)
        assert torch.equal(y, E.int8_matmul(q, s, wq, ws, None, dtype)) and torch.isfinite(y).all()
        _check_product(E, q, s, wq, ws, None, dtype)


@pytest.mark.parametrize("m", [1, 5, 70, 300])
def test_product_rows_inside_wider_matrices(E, m):
    A, sa, B, sb, bias = _operands(6, 2 * m, 400, 512)
    _check_product(E, A[::2, 64:364], sa[:m], B[100:301, 128:428], sb[:201], bias[:201], torch.bfloat16)


def test_product_of_a_nan_scale_is_a_nan_row(E):
    A, sa, B, sb, bias = _operands(7, 140, 200, 96)
    sa[3] = float("nan")
    Y = E.int8_matmul(A, sa, B, sb, bias)
    assert torch.isnan(Y[3]).all() and torch.isfinite(Y[:3]).all() and torch.isfinite(Y[4:]).all()


def test_no_tokens(E):
    from entropy_constrained_unbiased_b200.linear import int8_linear
    _, _, B, sb, bias = _operands(8, 1, 40, 64)
    Y = int8_linear(torch.empty((0, 64), device="cuda"), B, sb, bias)
    assert Y.shape == (0, 40)


@pytest.mark.parametrize("shape", [(64,), (1, 64), (2, 3, 64), (2, 0, 64)])
def test_linear_keeps_leading_dimensions_and_type(E, shape):
    from entropy_constrained_unbiased_b200.linear import int8_linear
    w = _x(9, 40, 64, torch.float32)
    wq, ws, _ = E.int8_quantize(w)
    x = torch.randn(shape, generator=torch.Generator().manual_seed(1)).half().cuda()
    y = int8_linear(x, wq, ws)
    assert y.shape == (*shape[:-1], 40) and y.dtype == torch.float16
    if y.numel():
        q, s, _ = E.int8_quantize(x.reshape(-1, 64))
        assert torch.equal(y.reshape(-1, 40), E.int8_matmul(q, s, wq, ws, None, torch.float16))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 300, 4099), (2, 65, 16384), (3, 129, 100), (5, 7, 33), (8, 1000, 520),
                                   (7, 9000, 64), (8, 40, 20000), (1, 33, 131072), (9, 100, 70), (40, 200, 1000)])
def test_linear_equals_its_two_steps(E, m, n, k, dtype):
    """One call gives what quantising and multiplying give, bit for bit, from few tokens (one kernel) to many."""
    w = _x(n, n, k, torch.float32)
    wq, ws, _ = E.int8_quantize(w)
    bias = torch.randn(n, generator=torch.Generator().manual_seed(2)).cuda()
    x = _x(m + k, m, k, dtype)
    if m > 2:
        x[1] = 0
        x[2, k // 2] = float("nan")
    q, s, _ = E.int8_quantize(x)
    for b in (None, bias):
        y, z = E.int8_linear(x, wq, ws, b), E.int8_matmul(q, s, wq, ws, b, dtype)
        assert y.dtype == dtype and torch.equal(y.nan_to_num(7.0), z.nan_to_num(7.0))
        assert torch.isnan(y).any() == (m > 2)
    off = torch.empty((m, k + 3), dtype=dtype, device="cuda")
    off[:, 3:] = x
    assert torch.equal(E.int8_linear(off[:, 3:], wq, ws).nan_to_num(7.0), E.int8_linear(x, wq, ws).nan_to_num(7.0))


@pytest.mark.parametrize("n,k", [(1, 777), (40, 777), (40, 33), (40, 1), (40, 768)])
def test_linear_with_dense_copies_of_the_weights(E, n, k):
    """Weights that lost their rows' padding on the way (a clone, a round trip through the host, a loaded state)."""
    from entropy_constrained_unbiased_b200.linear import int8_linear
    wq, ws, _ = E.int8_quantize(_x(9, n, k, torch.float32))
    x = _x(10, 5, k, torch.bfloat16)
    want = int8_linear(x, wq, ws)
    layer = torch.nn.Module()
    layer.register_buffer("weight", torch.zeros((n, k), dtype=torch.int8, device="cuda"))
    layer.load_state_dict({"weight": wq})
    for w in (wq.clone(memory_format=torch.contiguous_format), wq.cpu().cuda(), layer.weight):
        assert torch.equal(int8_linear(x, w, ws), want)


def test_linear_refuses_a_gradient(E):
    from entropy_constrained_unbiased_b200.linear import int8_linear
    wq, ws, _ = E.int8_quantize(_x(9, 40, 64, torch.float32))
    x = _x(1, 2, 64, torch.float32).requires_grad_()
    with pytest.raises(E.EcasqError):
        int8_linear(x, wq, ws)
    with torch.no_grad():
        int8_linear(x, wq, ws)


def test_linear_is_near_the_float_layer(E):
    """Each integer is off by at most half a step: |y - x W^T| <= sum of the two operands' rounding errors."""
    from entropy_constrained_unbiased_b200.linear import int8_linear
    x, w = _x(10, 30, 500, torch.float32), _x(11, 70, 500, torch.float32)
    wq, ws, _ = E.int8_quantize(w)
    y = _f64(int8_linear(x, wq, ws))
    X, Wt = _f64(x), _f64(w)
    ax, aw = np.abs(X).max(1, keepdims=True) / 254, np.abs(Wt).max(1, keepdims=True) / 254
    tol = ax * np.abs(Wt).sum(1) + np.abs(X).sum(1, keepdims=True) * aw.T + 500 * ax * aw.T
    assert np.all(np.abs(y - X @ Wt.T) <= tol * 1.001)


def test_overlapping_calls_and_graph_replay(E):
    """Calls on several streams at once, and a captured call replayed on new inputs, equal the plain calls."""
    ops = [_operands(20 + i, m, 512, 1024) for i, m in enumerate((1, 12, 90, 300))]
    want = [E.int8_matmul(A, sa, B, sb, bias) for A, sa, B, sb, bias in ops]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ops]
    got = []
    for _ in range(5):
        got = []
        for s, (A, sa, B, sb, bias) in zip(streams, ops):
            with torch.cuda.stream(s):
                got.append(E.int8_matmul(A, sa, B, sb, bias))
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    from entropy_constrained_unbiased_b200.linear import int8_linear
    wq, ws, _ = E.int8_quantize(_x(30, 256, 512, torch.float32))
    for m in (1, 40, 300):
        x = _x(31, m, 512, torch.bfloat16)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = int8_linear(x, wq, ws)
        x.copy_(_x(32, m, 512, torch.bfloat16))
        for _ in range(2):
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, int8_linear(x, wq, ws))


LONG_FEW = """
import torch
from entropy_constrained_unbiased_b200 import ecasq as E

for m, k in [(1, 49137), (1, 49152), (2, 24561), (2, 24576), (1, 49153), (1, 65536), (2, 32768)]:
    g = torch.Generator().manual_seed(k)
    rows = torch.zeros((m + 20, (k + 31) // 32 * 32), dtype=torch.int8)
    rows[:, :k] = torch.randint(-127, 128, (m + 20, k), generator=g, dtype=torch.int8)
    rows = rows.cuda()[:, :k]
    A, B, ones = rows[:m], rows[m:], torch.ones(20, device="cuda")
    want = (A.double() @ B.double().T).float()
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        scale = torch.full((m,), 2.0**-16, device="cuda")
        assert torch.equal(E.int8_matmul(A, scale, B, ones, None, dtype), (want * 2.0**-16).to(dtype)), (m, k, dtype)
        x = A.to(dtype)
        x[:, 0] = 127
        q, s, _ = E.int8_quantize(x)
        assert torch.equal(E.int8_linear(x, B, ones), E.int8_matmul(q, s, B, ones, None, dtype)), (m, k, dtype)
"""


def test_few_tokens_around_48_kb():
    """Tokens that need 48 KB of shared memory, just less and more, in a process whose first calls they are (a longer
    call before them would have raised the kernel's limit)."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", LONG_FEW], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]


def test_check_stalled_waits_for_every_stream(E):
    """The check returns after what runs on a stream that does not wait for the default one."""
    E.check_stalled()  # first: the library's symbols are loaded, which may wait by itself
    A, sa, B, sb, bias = _operands(40, 4096, 4096, 4096)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(200):  # tens of milliseconds
            E.int8_matmul(A, sa, B, sb, bias)
    E.check_stalled()
    assert side.query()
