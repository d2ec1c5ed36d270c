"""Refusals of the 8-bit operators, on the CPU: the C ABI's argument checks return before any CUDA call."""
import ctypes as C

import pytest
import torch

P16, ODD = C.c_void_p(1 << 20), C.c_void_p((1 << 20) + 8)  # never dereferenced
NULL = None


@pytest.fixture(scope="module")
def lib():
    from entropy_constrained_unbiased_b200 import build, ecasq
    build.build()
    return ecasq.load()


def test_quantize_arguments(lib):
    f = lib.ecasq_int8_quantize
    good = [P16, 0, 4, 100, 100, P16, 112, P16, P16, NULL]
    for at, bad in [(0, NULL), (1, 3), (1, -1), (2, -1), (2, 1 << 31), (3, 0), (3, 1 << 28), (4, 99), (5, NULL), (5, ODD),
                    (6, 104), (6, 96), (7, NULL), (8, NULL)]:
        args = list(good)
        args[at] = bad
        assert f(*args) == -1, (at, bad)
    assert f(NULL, 0, 0, 100, 100, NULL, 0, NULL, NULL, NULL) == 0  # no rows


def test_matmul_arguments(lib):
    f = lib.ecasq_int8_matmul
    good = [P16, 112, P16, P16, 112, P16, NULL, 4, 8, 100, P16, 1, 8, NULL]
    for at, bad in [(0, NULL), (0, ODD), (1, 104), (1, 96), (2, NULL), (3, NULL), (3, ODD), (4, 100), (4, 80), (5, NULL),
                    (7, -1), (7, 1 << 31), (8, 0), (8, 1 << 31), (9, 0), (9, 131073), (10, NULL), (11, 5), (12, 7)]:
        args = list(good)
        args[at] = bad
        assert f(*args) == -1, (at, bad)
    assert f(NULL, 0, NULL, NULL, 0, NULL, NULL, 0, 8, 100, NULL, 1, 8, NULL) == 0


def test_linear_arguments(lib):
    f = lib.ecasq_int8_linear
    good = [P16, 1, 100, P16, 112, P16, NULL, 40, 8, 100, P16, 8, P16, 1 << 20, NULL]
    for at, bad in [(0, NULL), (1, 4), (2, 99), (3, NULL), (3, ODD), (4, 104), (5, NULL), (7, -1), (8, 0), (9, 0), (9, 131073),
                    (10, NULL), (11, 7)]:
        args = list(good)
        args[at] = bad
        assert f(*args) == -1, (at, bad)
    need = lib.ecasq_int8_linear_workspace_size(40, 100)
    assert need >= 40 * (128 + 4)
    for at, bad in [(12, NULL), (12, ODD), (13, need - 1)]:
        args = list(good)
        args[at] = bad
        assert f(*args) == -3, (at, bad)
    assert f(NULL, 1, 100, NULL, 0, NULL, NULL, 0, 8, 100, NULL, 8, NULL, 0, NULL) == 0
    assert lib.ecasq_int8_linear_workspace_size(-1, 100) == 0 and lib.ecasq_int8_linear_workspace_size(4, 0) == 0


def test_checkpoint_arguments(lib):
    f = lib.ecasq_checkpoint8
    good = [P16, 0, 4, 100, 100, 7, NULL, P16, 128, P16, 16, NULL]
    for at, bad in [(0, NULL), (1, 3), (2, -1), (3, 0), (4, 99), (7, NULL), (7, ODD), (8, 112), (8, 96), (9, NULL), (9, ODD),
                    (10, 4), (10, 0)]:
        args = list(good)
        args[at] = bad
        assert f(*args) == -1, (at, bad)
    assert f(NULL, 0, 0, 100, 100, 7, NULL, NULL, 0, NULL, 0, NULL) == 0
    g = lib.ecasq_checkpoint8_restore
    good = [P16, 128, P16, 16, 4, 100, P16, 1, 100, NULL]
    for at, bad in [(0, NULL), (0, ODD), (1, 112), (2, NULL), (3, 8), (4, -1), (5, 0), (6, NULL), (7, 4), (8, 64)]:
        args = list(good)
        args[at] = bad
        assert g(*args) == -1, (at, bad)


def test_gradient_arguments(lib):
    f = lib.ecasq_checkpoint8_wgrad
    big = 1 << 40
    good = [P16, 1, 64, P16, 128, P16, 16, 4, 64, 100, P16, 1, 100, P16, big, NULL]
    for at, bad in [(0, NULL), (1, 3), (2, 63), (3, NULL), (3, ODD), (4, 112), (5, NULL), (6, 8), (7, -1), (8, 0), (8, 1 << 28),
                    (9, 0), (10, NULL), (11, 7), (12, 99)]:
        args = list(good)
        args[at] = bad
        assert f(*args) == -1, (at, bad)
    size = lib.ecasq_checkpoint8_wgrad_workspace_size
    assert size(P16, 1, 64, -1, 64, 100) == 0 and size(P16, 1, 64, 4, 0, 100) == 0 and size(P16, 9, 64, 4, 64, 100) == 0


def test_arrays_off_their_elements(lib):
    """Matrices of a type given at run time that start inside an element are refused."""
    for ty, off in [(0, 2), (0, 1), (1, 1), (2, 1)]:
        bad = C.c_void_p(P16.value + off)
        assert lib.ecasq_int8_quantize(bad, ty, 4, 100, 100, P16, 112, P16, P16, NULL) == -1
        assert lib.ecasq_int8_matmul(P16, 112, P16, P16, 112, P16, NULL, 4, 8, 100, bad, ty, 8, NULL) == -1
        for x, y in [(bad, P16), (P16, bad)]:
            assert lib.ecasq_int8_linear(x, ty, 100, P16, 112, P16, NULL, 40, 8, 100, y, 8, P16, 1 << 20, NULL) == -1
        assert lib.ecasq_checkpoint8(bad, ty, 4, 100, 100, 7, NULL, P16, 128, P16, 16, NULL) == -1
        assert lib.ecasq_checkpoint8_restore(P16, 128, P16, 16, 4, 100, bad, ty, 100, NULL) == -1
        for dy, dw in [(bad, P16), (P16, bad)]:
            assert lib.ecasq_checkpoint8_wgrad(dy, ty, 64, P16, 128, P16, 16, 4, 64, 100, dw, ty, 100, P16, 1 << 40,
                                               NULL) == -1


def test_gradient_workspace(lib):
    """Null, short and misaligned workspaces are refused: dY is copied into bf16 terms (float16, float32, rows off the
    16-byte boundary), or the sum over the tokens is split."""
    f, size = lib.ecasq_checkpoint8_wgrad, lib.ecasq_checkpoint8_wgrad_workspace_size
    for ty, ldy, t in [(0, 64, 4), (2, 64, 4), (1, 65, 4), (1, 64, 4096)]:
        need = size(P16, ty, ldy, t, 64, 100)
        assert need > 0
        for ws, have in [(NULL, need), (P16, need - 1), (ODD, need), (C.c_void_p(P16.value + 2), need)]:
            assert f(P16, ty, ldy, P16, 128, P16, 16, t, 64, 100, P16, 1, 100, ws, have, NULL) == -3, (ty, ldy, t, ws, have)


def test_no_cpu_path():
    from entropy_constrained_unbiased_b200 import ecasq as E
    from entropy_constrained_unbiased_b200.linear import checkpoint_linear, int8_linear
    x = torch.zeros((2, 32))
    q, s = torch.zeros((2, 32), dtype=torch.int8), torch.zeros(2)
    for call in (lambda: E.int8_quantize(x), lambda: E.int8_matmul(q, s, q, s), lambda: E.checkpoint8(x, 1),
                 lambda: E.checkpoint8_restore(q, q.view(torch.uint8)), lambda: int8_linear(x, q, s),
                 lambda: E.checkpoint8_wgrad(x, q, q.view(torch.uint8)), lambda: checkpoint_linear(x, x, seed=1), lambda: E.int8_linear(x, q, s)):
        with pytest.raises(E.EcasqError):
            call()


def test_int8_linear_refuses_gradients():
    """No operand's gradient is silently lost (looked at before the device)."""
    from entropy_constrained_unbiased_b200 import ecasq as E
    from entropy_constrained_unbiased_b200.linear import int8_linear
    x, w, s = torch.zeros((2, 32)), torch.zeros((2, 32), dtype=torch.int8), torch.zeros(2)
    grad = lambda t: t.clone().requires_grad_()
    for args in ((grad(x), w, s), (x, w, grad(s)), (x, w, s, grad(s)), (x, w, s.clone(), grad(s))):
        with pytest.raises(E.EcasqError, match="no gradient"):
            int8_linear(*args)
        with torch.no_grad(), pytest.raises(E.EcasqError, match="CUDA"):
            int8_linear(*args)


@pytest.mark.gpu
def test_binding_refusals():
    """Types, shapes, layouts and devices that the binding refuses before the library is called."""
    from entropy_constrained_unbiased_b200 import ecasq as E
    from entropy_constrained_unbiased_b200.linear import checkpoint_linear
    x = torch.zeros((4, 64), device="cuda")
    q, s, _ = E.int8_quantize(x)
    c, b = E.checkpoint8(x, 1)
    odd = torch.zeros((4, 33), dtype=torch.int8, device="cuda")
    calls = [
        lambda: E.int8_quantize(x.double()), lambda: E.int8_quantize(x[0]), lambda: E.int8_quantize(x.T[:, ::2]),
        lambda: E.int8_quantize(x[:1].expand(4, 64)), lambda: E.int8_quantize(x[:, :0]),
        lambda: E.int8_matmul(odd, s, odd, s), lambda: E.int8_matmul(q, s, q[:, :32], s), lambda: E.int8_matmul(q, s[:3], q, s),
        lambda: E.int8_matmul(q, s, q, s.double()), lambda: E.int8_matmul(q, s, q, s, s.bfloat16()),
        lambda: E.int8_matmul(q[:, 8:], s, q[:, 8:], s), lambda: E.int8_matmul(q, s, q[:0], s[:0]),
        lambda: E.int8_matmul(q, s.cpu(), q, s), lambda: E.int8_matmul(q, s, q, s, out_dtype=torch.float64),
        lambda: E.checkpoint8(x, torch.tensor([1])), lambda: E.checkpoint8(x, 1.5), lambda: E.checkpoint8(x, None), lambda: E.checkpoint8(x, torch.zeros(2, dtype=torch.int64, device="cuda")),
        lambda: E.checkpoint8_restore(c, b[:, :1]), lambda: E.checkpoint8_restore(c, b, torch.int8),
        lambda: E.checkpoint8_restore(odd, b), lambda: E.checkpoint8_wgrad(x[:3], c, b),
        lambda: E.checkpoint8_wgrad(x.double(), c, b), lambda: E.checkpoint8_wgrad(x, c, b, torch.int32),
        lambda: checkpoint_linear(x, x[:, :32], seed=1),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(E.EcasqError):
            call()
            pytest.fail(f"call {i} was not refused")
    wide = torch.zeros((2, 131104), dtype=torch.int8, device="cuda")
    with pytest.raises(E.EcasqError):
        E.int8_matmul(wide, s[:2], wide, s[:2])
