"""Refusals of the training operators, which need no GPU: every call here is turned
away on the host, before anything is launched."""

import ctypes

import pytest
import torch

import matrix_optimizers_sharded_amd as mo
from matrix_optimizers_sharded_amd import MatoptError, operators

FAKE = 0x10000
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3


def call(name, *args):
    return operators._call(name)(*args)


def error():
    return mo.load_library().mo_last_error().decode()


def refused(want, text, name, *args):
    assert call(name, *args) == want, (name, args, error())
    assert text in error(), (error(), text)


def test_group_rows_refuses():
    good = [FAKE, 8, 100, 7, FAKE, FAKE, None, 0, None]

    def bad(want, text, **at):
        a = list(good)
        for i, v in at.items():
            a[int(i[1:])] = v
        refused(want, text, "mo_group_rows", *a)

    bad(UNSUPPORTED, "4- or 8-byte", _1=2)
    bad(INVALID, "n must be", _2=-1)
    bad(INVALID, "n must be", _2=1 << 31)
    bad(INVALID, "number of keys", _3=0)
    bad(INVALID, "number of keys", _3=(1 << 26) + 1)
    bad(INVALID, "keys is NULL", _0=None)
    bad(INVALID, "order or offsets", _4=None)
    bad(INVALID, "order or offsets", _5=None)
    need = call("mo_group_rows_workspace_bytes", 100000, 7)
    assert need > 0 and call("mo_group_rows_workspace_bytes", 8192, 7) == 0
    assert call("mo_group_rows_workspace_bytes", -1, 7) == 0
    bad(WORKSPACE, "workspace is NULL", _2=100000)
    bad(WORKSPACE, "too small", _2=100000, _6=FAKE, _7=need - 1)
    bad(WORKSPACE, "aligned", _2=100000, _6=FAKE + 16, _7=need)


def test_embedding_refuses():
    look = [FAKE, 16, FAKE, 8, 5, 9, 16, 1, 1, 1.0, FAKE, None]
    grad = [FAKE, 16, FAKE, 8, 5, 9, 16, 1, 1, 1.0, FAKE, FAKE, 1 << 30, None]

    def bad(which, want, text, **at):
        a = list(look if which == "mo_embedding_lookup" else grad)
        for i, v in at.items():
            a[int(i[1:])] = v
        refused(want, text, which, *a)

    for f in ("mo_embedding_lookup", "mo_embedding_grad"):
        bad(f, INVALID, "pitch", _1=15)
        bad(f, UNSUPPORTED, "4- or 8-byte", _3=1)
        bad(f, INVALID, "n must be", _4=-3)
        bad(f, INVALID, "number of keys", _5=0)
        bad(f, INVALID, "dim must be", _6=0, _1=0)
        bad(f, UNSUPPORTED, "dtypes", _7=2)
        bad(f, UNSUPPORTED, "dtypes", _8=-1)
        bad(f, INVALID, "scale", _9=float("nan"))
        bad(f, INVALID, "tokens is NULL", _2=None)
        bad(f, INVALID, "is NULL", _0=None)
        bad(f, INVALID, "is NULL", _10=None)
    bad("mo_embedding_grad", WORKSPACE, "workspace is NULL", _11=None)
    bad("mo_embedding_grad", WORKSPACE, "too small", _12=64)
    assert call("mo_embedding_lookup", FAKE, 16, None, 8, 0, 9, 16, 1, 1, 1.0, None, None) == 0


def test_experts_refuse():
    def args(name, **at):
        a = dict(A=FAKE, lda=64, B=FAKE, ldb=64, off=FAKE, e=3, n=10, k=64, m=64, dt=1, out=1, C=FAKE)
        a.update(at)
        head = [a["A"], a["lda"], a["B"]] + ([a["ldb"]] if name == "mo_expert_weight_grad" else [])
        return head + [a["off"], a["e"], a["n"], a["k"], a["m"], a["dt"], a["out"], a["C"], None]

    for f in ("mo_expert_matmul", "mo_expert_input_grad", "mo_expert_weight_grad"):
        for want, text, at in ((UNSUPPORTED, "dtypes", dict(dt=3)), (UNSUPPORTED, "dtypes", dict(out=9)),
                               (UNSUPPORTED, "fp32 operands", dict(dt=0, out=1)),
                               (INVALID, "experts must be", dict(e=0)), (INVALID, "experts must be", dict(e=1025)),
                               (INVALID, "n must be", dict(n=-1)), (INVALID, "n must be", dict(n=1 << 31)),
                               (INVALID, "k and m", dict(k=0)), (INVALID, "k and m", dict(m=(1 << 20) + 1)),
                               (INVALID, "pitch", dict(lda=63)), (INVALID, "pitch", dict(lda=(1 << 20) + 1)),
                               (INVALID, "offsets", dict(off=None)), (INVALID, "result", dict(C=None)),
                               (INVALID, "is NULL", dict(A=None)), (INVALID, "is NULL", dict(B=None))):
            refused(want, text, f, *args(f, **at))
    refused(INVALID, "pitch", "mo_expert_weight_grad", *args("mo_expert_weight_grad", ldb=63))
    refused(INVALID, "result", "mo_expert_weight_grad", *args("mo_expert_weight_grad", n=0, A=None, B=None, C=None))
    assert call("mo_expert_matmul", *args("mo_expert_matmul", n=0, A=None, C=None)) == 0


def test_distill_refuses():
    def args(name, **at):
        a = dict(x=FAKE, ld=100, lse=FAKE, ids=FAKE, ib=8, t=FAKE, rg=FAKE, n=4, v=100, k=8, dt=0, tau=1.0, loss=FAKE,
                 grad=0x90000, ldg=100)
        a.update(at)
        a = {k: (ctypes.c_float(v) if k == "tau" else v) for k, v in a.items()}
        shape = [a["n"], a["v"], a["k"], a["dt"], a["tau"]]
        if name == "mo_distill_forward":
            return [a["x"], a["ld"], a["ids"], a["ib"], a["t"]] + shape + [a["loss"], a["lse"], None]
        if name == "mo_distill_backward":
            return [a["x"], a["ld"], a["lse"], a["ids"], a["ib"], a["t"], a["rg"]] + shape + [a["grad"], a["ldg"], None]
        return ([a["x"], a["ld"], a["ids"], a["ib"], a["t"], a["rg"]] + shape +
                [a["loss"], a["lse"], a["grad"], a["ldg"], None])

    every = ("mo_distill_forward", "mo_distill_backward", "mo_distill_forward_backward")
    for f in every:
        for want, text, at in ((UNSUPPORTED, "dtype", dict(dt=2)), (UNSUPPORTED, "indices", dict(ib=2)),
                               (INVALID, "n must be", dict(n=-1)), (INVALID, "vocab", dict(v=0)),
                               (INVALID, "teacher entries", dict(k=0)), (INVALID, "teacher entries", dict(k=1025)),
                               (INVALID, "temperature", dict(tau=0.0)), (INVALID, "temperature", dict(tau=-1.0)),
                               (INVALID, "temperature", dict(tau=float("inf"))),
                               (INVALID, "temperature", dict(tau=float("nan"))), (INVALID, "pitch", dict(ld=99)),
                               (INVALID, "NULL", dict(x=None)), (INVALID, "NULL", dict(ids=None)),
                               (INVALID, "NULL", dict(t=None)), (INVALID, "NULL", dict(lse=None))):
            refused(want, text, f, *args(f, **at))
        assert call(f, *args(f, n=0)) == 0
    for f in every[1:]:
        refused(INVALID, "pitch", f, *args(f, ldg=99))
        refused(INVALID, "NULL", f, *args(f, grad=None))
        refused(INVALID, "NULL", f, *args(f, rg=None))
    refused(INVALID, "grad must not be logits", every[2], *args(every[2], grad=FAKE))


def test_the_binding_refuses():
    cpu = torch.zeros(4, 6)
    tok = torch.zeros(4, dtype=torch.int64)
    off = torch.zeros(3, dtype=torch.int32)
    w = torch.zeros(2, 5, 6)
    ids = torch.zeros(4, 3, dtype=torch.int64)
    t = torch.zeros(4, 3)
    for f in (lambda: mo.group_rows(tok, 5), lambda: mo.embedding_lookup(cpu, tok),
              lambda: mo.embedding_grad(cpu, tok, 9), lambda: mo.expert_matmul(cpu, w, off),
              lambda: mo.expert_input_grad(torch.zeros(4, 5), w, off),
              lambda: mo.expert_weight_grad(torch.zeros(4, 5), cpu, off), lambda: mo.distill_forward(cpu, ids, t)):
        with pytest.raises(MatoptError, match="CUDA"):
            f()
    for text, f in (("expected int32 or int64", lambda: mo.group_rows(tok.float(), 5)),
                    ("contiguous vector", lambda: mo.group_rows(ids, 5)),
                    ("two dimensions", lambda: mo.embedding_lookup(w, tok)),
                    ("unit column stride", lambda: mo.embedding_lookup(cpu.t(), tok)),
                    ("rows overlap", lambda: mo.embedding_lookup(cpu[:1].expand(4, 6), tok)),
                    ("one for each row", lambda: mo.embedding_grad(cpu, tok[:3], 9)),
                    ("contiguous tensor", lambda: mo.expert_matmul(cpu, w.transpose(1, 2), off)),
                    ("offsets: expected 3", lambda: mo.expert_matmul(cpu, w, off[:2])),
                    ("int32 vector", lambda: mo.expert_matmul(cpu, w, off.long())),
                    ("expected 6 columns", lambda: mo.expert_matmul(cpu[:, :5], w, off)),
                    ("expected 5 columns", lambda: mo.expert_input_grad(cpu, w, off)),
                    ("one dtype", lambda: mo.expert_matmul(cpu.bfloat16(), w, off)),
                    ("expected 4 rows", lambda: mo.expert_weight_grad(cpu, cpu[:3], off)),
                    ("one shape", lambda: mo.distill_forward(cpu, ids, t[:, :2])),
                    ("float32", lambda: mo.distill_forward(cpu, ids, t.bfloat16())),
                    ("unsupported dtype", lambda: mo.distill_forward(cpu.half(), ids, t)),
                    ("temperature", lambda: mo.distill_forward(cpu, ids, t, temperature=0.0)),
                    ("row_grad", lambda: mo.distill_forward_backward(cpu, ids, t, torch.zeros(3))),
                    ("lse", lambda: mo.distill_backward(cpu, torch.zeros(4, 1), ids, t, torch.zeros(4)))):
        with pytest.raises(MatoptError, match=text):
            f()


def test_expert_products_refuse_rows_past_32_bits():
    """Tile counts round a segment's rows up, within 32 bits."""
    for name, a in (("mo_expert_matmul", [FAKE, 8, FAKE, FAKE, 1, None, 8, 8, 1, 1, FAKE, None]),
                    ("mo_expert_input_grad", [FAKE, 8, FAKE, FAKE, 1, None, 8, 8, 1, 1, FAKE, None]),
                    ("mo_expert_weight_grad", [FAKE, 8, FAKE, 8, FAKE, 1, None, 8, 8, 1, 1, FAKE, None])):
        for n in ((1 << 31) - 1023, (1 << 31) - 1, 1 << 31, -1):
            b = [n if v is None and i in (5, 6) else v for i, v in enumerate(a)]
            refused(INVALID, "n must be", name, *b)


def test_distill_refuses_a_gradient_over_the_logits():
    """The kernels read a row's logits again after they have stored its gradient."""
    n, v = 4, 100
    shape = [n, v, 8, 0, ctypes.c_float(1.0)]

    def args(name, logits, ld, grad, ldg):
        if name == "mo_distill_backward":
            return [logits, ld, 0x1000, 0x2000, 8, 0x3000, 0x4000] + shape + [grad, ldg, None]
        return [logits, ld, 0x2000, 8, 0x3000, 0x4000] + shape + [0x5000, 0x6000, grad, ldg, None]

    at = 0x100000
    for f in ("mo_distill_backward", "mo_distill_forward_backward"):
        for logits, ld, grad, ldg in ((at, 100, at, 100), (at, 100, at + 400, 100), (at + 1596, 100, at, 100),
                                      (at, 100, at + 1596, 250), (at, 250, at + 396, 250), (at + 396, 250, at, 250),
                                      (at, 1 << 61, at + 4, 100)):
            refused(INVALID, "grad must not be logits", f, *args(f, logits, ld, grad, ldg))
        # side by side, and one behind the other: past this check (and then, without a GPU or
        # with no rows, no further)
        for logits, ld, grad, ldg in ((at, 250, at + 400, 250), (at + 600, 250, at, 250), (at, 100, at + 1600, 100)):
            a = args(f, logits, ld, grad, ldg)
            if not torch.cuda.is_available():
                assert call(f, *a) != INVALID, error()


def test_distill_refuses_temperatures_without_a_reciprocal():
    for tau in (2.0 ** -127, 2.0 ** -149):
        refused(INVALID, "temperature", "mo_distill_forward", FAKE, 100, FAKE, 8, FAKE, 4, 100, 8, 0, tau, FAKE, FAKE, None)
        refused(INVALID, "temperature", "mo_distill_backward", FAKE, 100, FAKE, FAKE, 8, FAKE, FAKE, 4, 100, 8, 0, tau,
                FAKE << 8, 100, None)
        refused(INVALID, "temperature", "mo_distill_forward_backward", FAKE, 100, FAKE, 8, FAKE, FAKE, 4, 100, 8, 0, tau,
                FAKE, FAKE, FAKE << 8, 100, None)


def test_results_over_inputs_are_refused():
    """Other blocks still read what one block overwrites."""
    at, text = 0x100000, "must not overlap an input"
    for out in (at, at + 196, at - 36):                      # 50 int32 keys, 10 result words
        refused(INVALID, text, "mo_group_rows", at, 4, 50, 9, FAKE, out, None, 0, None)
    refused(INVALID, text, "mo_group_rows", at, 8, 50, 9, at + 392, FAKE, None, 0, None)
    # a table of 9 rows of 16 bf16 values 20 apart (352 bytes), 5 tokens of 8 bytes
    for out in (at, at + 350, at - 159):
        refused(INVALID, text, "mo_embedding_lookup", at, 20, FAKE, 8, 5, 9, 16, 1, 1, 1.0, out, None)
    refused(INVALID, text, "mo_embedding_lookup", FAKE, 20, at, 8, 5, 9, 16, 1, 1, 1.0, at + 36, None)
    for out in (at, at + 190, at - 286):                     # 5 rows 20 apart (192 bytes), 288 bytes of result
        refused(INVALID, text, "mo_embedding_grad", at, 20, FAKE, 8, 5, 9, 16, 1, 1, 1.0, out, FAKE, 1 << 30, None)
    refused(INVALID, text, "mo_embedding_grad", FAKE, 20, at, 8, 5, 9, 16, 1, 1, 1.0, at + 36, FAKE, 1 << 30, None)
    # 10 rows of 64 bf16 values, 3 experts of 64 x 64, offsets of 16 bytes
    far, off = 0x900000, 0x800000
    for name, w_rows in (("mo_expert_matmul", 192), ("mo_expert_input_grad", 192)):
        for out in (at, at + 1278, at - 1278, far, far + 128 * w_rows - 2, off, off + 14):
            refused(INVALID, text, name, at, 64, far, off, 3, 10, 64, 64, 1, 1, out, None)
    for out in (at, at + 1278, at - 24574, far, off, off + 14):
        refused(INVALID, text, "mo_expert_weight_grad", at, 64, far, 64, off, 3, 10, 64, 64, 1, 1, out, None)
    if not torch.cuda.is_available():      # apart: past this check, and no further without a GPU
        for out in (at + 1280, at - 1280, far - 1280, far + 24576, off + 16):
            assert call("mo_expert_matmul", at, 64, far, off, 3, 10, 64, 64, 1, 1, out, None) != INVALID, error()


def test_sign_calls_refuse_more_than_a_launch_holds():
    """2^24 blocks of 256 threads are 2^32 threads, of which only the remainder would run."""
    lib = mo.load_library()
    for numel in ((1 << 40) + 1, 1 << 41):
        for rc in (lib.sign_pack(FAKE, 0, numel, FAKE, None), lib.sign_pack_batched(FAKE, 1, 2, numel, numel, FAKE, None),
                   lib.sign_vote(FAKE, 3, numel, FAKE, None, None), lib.sign_unpack(FAKE, numel, 1, FAKE, None),
                   lib.sign_apply(FAKE, numel, 1, FAKE, 0.5, None)):
            assert rc == INVALID and "too large" in error(), (numel, rc, error())
