"""Products by expert under tables of offsets that are not ascending: every row of the
results is written, by one expert, whatever the table holds."""

import pytest
import torch

import matrix_optimizers_sharded_amd as mo
from gpu_util import say
from test_gpu_operators import BF16, F32, U32, close, generator, u

pytestmark = pytest.mark.gpu

N = 1500
TABLES = {
    "descends": [0, 750, 0, 750, 0, 750, N],
    "backwards": list(range(N, -1, -250)),
    "outside": [-7, 300, 1 << 30, 200, -(1 << 31), N + 1],
    "one dip": [10, 600, 599, 900, 1400],
    "many, with dips past 64": [(37 * i) % N if i % 5 == 0 else min(N, 8 * i) for i in range(150)],
    "all at the end": [N] * 4,
    "ascending": [3, 3, 500, 500, 1499],
}


def owners(table):
    """The expert of every row, -1 for none: a bound below an earlier one counts as that."""
    top, last, expert = 0, 0, [-1] * N
    for e, o in enumerate(table):
        top = max(top, min(max(o, 0), N))
        if e > 0:
            expert[last:top] = [e - 1] * (top - last)
        last = top
    return torch.tensor(expert)


# widths that take the split sum, the small tile, the middle one and the large one
WIDTHS = [(520, 64), (64, 1160), (264, 2100), (65, 129), (1024, 16400)]


@pytest.mark.parametrize("k,m", WIDTHS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("name", TABLES)
def test_offsets_that_do_not_ascend(gpu, name, dtype, k, m):
    if dtype == F32 and m > 4000:
        m = 2100
    table = TABLES[name]
    say(f"experts: offsets that {name}, {k} x {m} {dtype}")
    gen = generator(gpu, k)
    e_all = len(table) - 1
    off = torch.tensor(table, device=gpu, dtype=torch.int64).to(torch.int32)
    x = torch.randn(N, k, generator=gen, device=gpu).to(dtype)
    dy = torch.randn(N, m, generator=gen, device=gpu).to(dtype)
    w = torch.randn(e_all, m, k, generator=gen, device=gpu).to(dtype)
    nan = float("nan")
    y = mo.expert_matmul(x, w, off, out=torch.full((N, m), nan, device=gpu, dtype=dtype))
    dx = mo.expert_input_grad(dy, w, off, out=torch.full((N, k), nan, device=gpu, dtype=dtype))
    dw = mo.expert_weight_grad(dy, x, off, out=torch.full((e_all, m, k), nan, device=gpu, dtype=dtype))
    who = owners(table).to(gpu)
    want = [torch.zeros(t.shape, dtype=torch.float64, device=gpu) for t in (y, dx)]
    size = [torch.zeros_like(t) for t in want]

    def check(what, got, t, s, length):
        # a matrix instruction may round every product and every sum: two roundings a term
        close(got, t, s * 2 * (length + 1) * U32 + t.abs() * u(dtype) * 1.01, what)

    for e in range(e_all):
        r = torch.nonzero(who == e)[:, 0]
        a, b, c = x[r].double(), dy[r].double(), w[e].double()
        want[0][r], size[0][r] = a @ c.t(), a.abs() @ c.abs().t()
        want[1][r], size[1][r] = b @ c, b.abs() @ c.abs()
        lo, hi = (min(max(o, 0), N) for o in table[e:e + 2])
        a, b = x[lo:max(lo, hi)].double(), dy[lo:max(lo, hi)].double()
        check(f"dw of expert {e}", dw[e], b.t() @ a, b.abs().t() @ a.abs(), N)
    check("y", y, want[0], size[0], k)
    check("dx", dx, want[1], size[1], m)
    again = mo.expert_matmul(x, w, off), mo.expert_input_grad(dy, w, off), mo.expert_weight_grad(dy, x, off)
    for a, b in zip((y, dx, dw), again):
        assert torch.equal(a, b)
