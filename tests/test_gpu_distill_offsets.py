"""The distillation loss on logits with a large common offset, and on rows that hold one
value only (a row that is masked whole, with whatever value the mask has).

softmax does not see a common offset: loss and gradient are those of the row without it."""

import math

import pytest
import torch

import matrix_optimizers_sharded_amd as mo
from gpu_util import say
from test_gpu_operators import BF16, F32, F64, U32, close, distill_exact, generator, u

pytestmark = pytest.mark.gpu

LENGTHS = [1000, 40000, 131080, 140000]    # held by a block for one type or both, and read twice


def teacher_rows(gpu, n, v, k, seed):
    gen = generator(gpu, seed)
    idx = torch.stack([torch.randperm(v, generator=gen, device=gpu)[:k] for _ in range(n)])
    t = torch.randn(n, k, generator=gen, device=gpu) * 4
    idx[torch.rand(n, k, generator=gen, device=gpu) < 0.2] = -1
    idx[0] = -1                     # a row that the loss leaves out
    return idx, t, torch.rand(n, generator=gen, device=gpu) + 0.5


def shifted(gpu, v, dtype, unit, offset, seed):
    """Logits that are whole multiples of `unit`, without and with the offset, exactly."""
    gen = generator(gpu, seed)
    x = torch.randint(0, 64, (4, v), generator=gen, device=gpu).to(F64) * unit
    plain, moved = x.to(dtype), (x + offset).to(dtype)
    assert torch.equal(plain.to(F64), x) and torch.equal(moved.to(F64), x + offset)
    return plain, moved


# multiples of `unit`, an offset that keeps them exact in the type, a temperature of the unit's order
OFFSETS = [(F32, 0.125, 2.0 ** 17, 1.0), (F32, 0.125, -2.0 ** 17, 1.7), (F32, 2.0 ** 11, 2.0 ** 33, 5000.0),
           (BF16, 1.0, 128.0, 5.0), (BF16, 1024.0, 2.0 ** 17, 1024.0), (BF16, 1024.0, -2.0 ** 17, 1700.0)]


@pytest.mark.parametrize("v", LENGTHS)
@pytest.mark.parametrize("dtype,unit,offset,tau", OFFSETS)
def test_a_common_offset_changes_nothing(gpu, dtype, unit, offset, tau, v):
    """The differences from the row's maximum are exact here, and equal: so is every bit of
    the loss and of the gradient in one pass."""
    say(f"distill offset {offset} v={v} {dtype}")
    plain, moved = shifted(gpu, v, dtype, unit, offset, v)
    idx, t, rg = teacher_rows(gpu, 4, v, 9, v + 1)
    loss, lse, grad = mo.distill_forward_backward(plain, idx, t, rg, temperature=tau)
    loss2, lse2, grad2 = mo.distill_forward_backward(moved, idx, t, rg, temperature=tau)
    assert torch.equal(loss, loss2) and torch.equal(grad, grad2)
    only = mo.distill_forward(moved, idx, t, temperature=tau)
    assert torch.equal(only[0], loss2) and torch.equal(only[1], lse2)
    # lse: the maximum by the temperature (two roundings), the logarithm, and their sum
    tau32 = float(torch.tensor(tau, dtype=F32))
    want = torch.logsumexp(moved.double() / tau32, 1)
    close(lse2, want, 4 * U32 * (want.abs() + moved.double().abs().amax(1) / tau32) + 1e-4, "lse")


def constant_tolerance(tau, t, k, q, whole, grad, rg, dtype):
    """A row of one value: every exponential is 1 exactly, their sum is exact, and what is
    left are the teacher's roundings, a logarithm's, and a handful of products."""
    rt = (3 * float(t.amax() - t.amin()) / tau * 1.4427 + 4 + k) * U32
    g = tau * rg.double()[:, None]
    tol_loss = tau * tau * (2 * rt + 8 * U32) * (16 + float(t.amax() - t.amin()) / tau)
    return tol_loss, g * (q * 8 * U32 + whole * (2 * rt + 4 * U32)) + grad.abs() * u(dtype) * 1.01


def constant_rows(gpu, v, dtype, value, tau):
    x = torch.full((4, v), value, dtype=F64, device=gpu).to(dtype)
    idx, t, rg = teacher_rows(gpu, 4, v, 9, v)
    tau32 = float(torch.tensor(tau, dtype=F32))
    # the definition does not depend on the value
    loss, _, grad, q, whole = distill_exact(torch.zeros_like(x), idx, t, rg, tau32)
    tol = constant_tolerance(tau32, t, 9, q, whole, grad, rg, dtype)
    return x, idx, t, rg, tau32, loss, grad, tol


VALUES = [1e4, -1e9, 1e10, -1e30, "lowest", "highest"]


def value_of(value, dtype):
    if isinstance(value, str):
        return torch.finfo(dtype).min if value == "lowest" else torch.finfo(dtype).max
    return value


@pytest.mark.parametrize("tau", [0.5, 1.0, 1.7, 2.0])
@pytest.mark.parametrize("value", VALUES)
@pytest.mark.parametrize("v", LENGTHS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_of_one_value(gpu, dtype, v, value, tau):
    value = value_of(value, dtype)
    x, idx, t, rg, tau32, want_loss, want_grad, tol = constant_rows(gpu, v, dtype, value, tau)
    loss, lse, grad = mo.distill_forward_backward(x, idx, t, rg, temperature=tau)
    only = mo.distill_forward(x, idx, t, temperature=tau)
    assert torch.equal(only[0], loss) and torch.equal(only[1], lse)
    close(loss, want_loss, tol[0], "loss")
    close(grad, want_grad, tol[1], "gradient in one pass")
    assert float(loss[0]) == 0 and not grad[0].any()
    want = float(x[0, 0].double()) / tau32 + math.log(v)
    if abs(want) > torch.finfo(F32).max:
        assert bool((lse == math.copysign(math.inf, want)).all())
    else:
        close(lse, torch.full((4,), want, dtype=F64, device=gpu), torch.tensor(abs(want) * 4 * U32, device=gpu), "lse")


@pytest.mark.parametrize("tau", [0.5, 1.0, 1.7, 2.0])
@pytest.mark.parametrize("value", VALUES)
@pytest.mark.parametrize("v", LENGTHS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradient_from_lse_of_rows_of_one_value(gpu, dtype, v, value, tau):
    value = value_of(value, dtype)
    x, idx, t, rg, tau32, _, want, tol = constant_rows(gpu, v, dtype, value, tau)
    _, lse = mo.distill_forward(x, idx, t, temperature=tau)
    grad = mo.distill_backward(x, lse, idx, t, rg, temperature=tau)
    close(grad, want, tol[1], "gradient from lse")
    assert not grad[0].any()


@pytest.mark.parametrize("v", LENGTHS)
@pytest.mark.parametrize("dtype,unit,offset,tau", OFFSETS + [(F32, 0.125, 900.0, 1.0), (F32, 0.125, -1100.0, 1.0)])
def test_gradient_from_lse_with_an_offset(gpu, dtype, unit, offset, tau, v):
    """Where lse is below 1024 in size, its own rounding and that of x / tau are an error of the
    exponent; beyond, the result is as exact as without an offset."""
    say(f"distill_backward offset {offset} v={v} {dtype}")
    plain, moved = shifted(gpu, v, dtype, unit, offset, v)
    idx, t, rg = teacher_rows(gpu, 4, v, 9, v + 1)
    tau32 = float(torch.tensor(tau, dtype=F32))
    _, _, want, q, whole = distill_exact(plain, idx, t, rg, tau32)
    _, lse = mo.distill_forward(moved, idx, t, temperature=tau)
    grad = mo.distill_backward(moved, lse, idx, t, rg, temperature=tau)
    reach = 63 * unit / tau * 1.4427
    rt = (3 * float(t.amax() - t.amin()) / tau * 1.4427 + 4 + 9) * U32
    rq = (6 * reach + 8 + v / 256 + 32) * U32       # a sum by 256 threads and one exponential
    low = lse.double().abs() < 1024
    rq = rq + torch.where(low, 4 * U32 * (lse.double().abs() + moved.double().abs().amax(1) / tau) * 1.4427, 0.0)
    g = tau * rg.double()[:, None]
    tol = g * (q * (rq[:, None] + 4 * U32) + whole * (2 * rt + 4 * U32)) + want.abs() * u(dtype) * 1.01
    close(grad, want, tol, "gradient from lse")


@pytest.mark.parametrize("dtype,tau", [(BF16, 0.25), (F32, 0.5), (F32, 0.9), (F32, 1.0), (F32, 1e-25), (F32, 2.0 ** -126)])
def test_losses_near_the_ends_of_their_type(gpu, dtype, tau):
    """A teacher that asks for logits of the type's lowest value, where the loss is as large
    as they are, times tau; and temperatures whose square is not a float."""
    tau32 = float(torch.tensor(tau, dtype=F32))
    x = torch.randn(3, 3000, generator=generator(gpu, 5), device=gpu).to(dtype)
    if tau > 0.1:
        x[:, 100:] = torch.finfo(dtype).min
    idx = torch.arange(95, 104, device=gpu).expand(3, 9).contiguous()
    t = torch.randn(3, 9, generator=generator(gpu, 6), device=gpu)
    loss, _ = mo.distill_forward(x, idx, t, temperature=tau)
    d = t.double() - t.double().amax(1, keepdim=True)
    away = torch.gather(x, 1, idx).double() - x.double().amax(1, keepdim=True)
    p = torch.softmax(d / tau32, 1)
    log_q = torch.log_softmax(x.double() / tau32, 1)
    assert bool(torch.isfinite(log_q).all())
    log_p = torch.log_softmax(d / tau32, 1)
    want = tau32 * tau32 * torch.where(p > 0, p * (log_p - torch.gather(log_q, 1, idx)), 0.0).sum(1)
    assert bool((want > 0).all()) and float(want.max()) < torch.finfo(F32).max
    # The sum's terms are off by the rounding of their weight (an exponent of d / tau, three
    # roundings of its size), of the sums of 9, and ten more; a weight below fp32's smallest
    # may be lost.
    rt = torch.where(p > 1e-38, 3 * (d / tau32).abs() * 1.4427 * U32, 1.0)
    size = (p * (d - away).abs() * (rt + (rt * p).sum(1, keepdim=True) + 32 * U32)).sum(1) * tau32
    close(loss, want, size + tau32 * tau32 * 64 * U32 * 16, "loss")
