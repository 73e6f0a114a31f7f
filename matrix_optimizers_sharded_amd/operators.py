"""The training operators around the owner-local step: grouping of rows by key, the
embedding table's lookup and gradient, products grouped by expert with both gradients,
and the distillation loss against a teacher's top logits with its gradient.

Argument marshalling only, as in binding.py: checks, result tensors (unless given as
out), raw pointers and torch's current stream.  The definitions are in
include/matopt.h.  Every call only enqueues work, so it can be captured into a graph;
there a call that takes a workspace is given one that has already served a call of the same
sizes and that lives as long as the graph, and calls that share a workspace, replays among
them, are ordered on one stream.  Rows of two-dimensional inputs may be padded
(any row pitch, unit column stride); results are contiguous and overlap no input.  No call
differentiates itself: the gradients are calls of their own.
"""

import ctypes
import functools

import torch

from .binding import MO_BF16, MO_F32, MatoptError, Workspace, load_library

_CODE = {torch.float32: MO_F32, torch.bfloat16: MO_BF16}
_INT = {torch.int32: 4, torch.int64: 8}
_fn = {}


def _call(name):
    f = _fn.get(name)
    if f is None:
        lib = load_library()
        P, I32, I64, SZ, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
        types = {
            "mo_group_rows_workspace_bytes": [I64, I64],
            "mo_group_rows": [P, I32, I64, I64, P, P, P, SZ, P],
            "mo_embedding_lookup": [P, I64, P, I32, I64, I64, I64, I32, I32, F, P, P],
            "mo_embedding_grad_workspace_bytes": [I64, I64, I64],
            "mo_embedding_grad": [P, I64, P, I32, I64, I64, I64, I32, I32, F, P, P, SZ, P],
            "mo_expert_matmul": [P, I64, P, P, I32, I64, I64, I64, I32, I32, P, P],
            "mo_expert_input_grad": [P, I64, P, P, I32, I64, I64, I64, I32, I32, P, P],
            "mo_expert_weight_grad": [P, I64, P, I64, P, I32, I64, I64, I64, I32, I32, P, P],
            "mo_distill_forward": [P, I64, P, I32, P, I64, I64, I64, I32, F, P, P, P],
            "mo_distill_backward": [P, I64, P, P, I32, P, P, I64, I64, I64, I32, F, P, I64, P],
            "mo_distill_forward_backward": [P, I64, P, I32, P, P, I64, I64, I64, I32, F, P, P, P, I64, P],
        }
        f = getattr(lib, name)
        f.argtypes = types[name]
        f.restype = SZ if name.endswith("_bytes") else I32
        _fn[name] = f
    return f


@functools.lru_cache(maxsize=256)
def _workspace_bytes(name, *sizes):
    """A workspace's size, which depends on these sizes alone."""
    return _call(name)(*sizes)


def _run(name, dev, *args):
    """One C call on dev's current stream, with dev current."""
    f = _fn.get(name) or _call(name)
    i = dev.index
    stream = torch._C._cuda_getCurrentRawStream(i)
    if torch._C._cuda_getDevice() == i:
        rc = f(*args, stream)
    else:
        with torch.cuda.device(dev):
            rc = f(*args, stream)
    if rc != 0:
        raise MatoptError(rc, load_library().mo_last_error().decode(errors="replace"))


def _bad(msg):
    raise MatoptError(-1, msg)


def _float(t, name):
    c = _CODE.get(t)
    if c is None:
        raise MatoptError(-2, f"{name}: unsupported dtype {t}")
    return c


def _int(t, name):
    c = _INT.get(t.dtype)
    if c is None:
        raise MatoptError(-2, f"{name}: expected int32 or int64, got {t.dtype}")
    if t.dim() != 1 or not t.is_contiguous():
        _bad(f"{name}: expected a contiguous vector")
    return c


def _device(first, *rest):
    """The one CUDA device that all tensors are on."""
    d = first.device
    if d.type != "cuda":
        _bad(f"expected CUDA tensors, got one on {d}")
    for t in rest:
        if t is not None and t.device != d:
            _bad(f"all tensors must be on one CUDA device, got {d} and {t.device}")
    return d


def _rows(t, name):
    """Row pitch of a two-dimensional tensor with unit column stride."""
    if t.dim() != 2:
        _bad(f"{name}: expected two dimensions, got {t.dim()}")
    n, w = t.shape
    s0, s1 = t.stride()
    if s1 != 1 and w > 1:
        _bad(f"{name}: expected unit column stride")
    if n <= 1:
        return w   # the pitch of a single row says nothing
    if s0 < w:
        _bad(f"{name}: rows overlap (pitch {s0}, width {w})")
    return s0


def _result(out, shape, dtype, dev, name):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if tuple(out.shape) != shape or out.dtype != dtype or out.device != dev or not out.is_contiguous():
        _bad(f"{name}: expected a contiguous {dtype} tensor of shape {shape} on {dev}")
    return out


def _scratch(workspace, dev, nbytes):
    if nbytes == 0:
        return None, None, 0
    buf = (workspace or Workspace(dev)).get(nbytes)
    if buf.device != dev:
        _bad(f"the workspace is on {buf.device}, the tensors on {dev}")
    return buf, buf.data_ptr(), buf.numel()


def group_rows(keys, num_keys, order=None, offsets=None, workspace=None):
    """Stable grouping of rows by key: (order, offsets), both int32.  order[p] is the row
    at position p; key v's rows are positions offsets[v] .. offsets[v + 1] - 1.  Rows
    with a key outside [0, num_keys) come last, from offsets[num_keys] on."""
    kb = _int(keys, "keys")
    dev = _device(keys)
    n, num_keys = keys.numel(), int(num_keys)
    if not 1 <= num_keys <= 1 << 26:
        _bad("the number of keys must be in [1, 2^26]")
    order = _result(order, (n,), torch.int32, dev, "order")
    offsets = _result(offsets, (num_keys + 1,), torch.int32, dev, "offsets")
    buf, ws, nb = _scratch(workspace, dev, _workspace_bytes("mo_group_rows_workspace_bytes", n, num_keys))
    _run("mo_group_rows", dev, keys.data_ptr(), kb, n, num_keys, order.data_ptr(), offsets.data_ptr(), ws, nb)
    return order, offsets


def embedding_lookup(table, tokens, scale=1.0, out_dtype=None, out=None):
    """scale * table[tokens] (n x dim); zeros where the token lies outside the table."""
    ld, tb = _rows(table, "table"), _int(tokens, "tokens")
    dev = _device(table, tokens)
    (vocab, dim), n = table.shape, tokens.numel()
    out_dtype = out_dtype or (out.dtype if out is not None else table.dtype)
    code, oc = _float(table.dtype, "table"), _float(out_dtype, "out")
    out = _result(out, (n, dim), out_dtype, dev, "out")
    _run("mo_embedding_lookup", dev, table.data_ptr(), ld, tokens.data_ptr(), tb, n, vocab, dim, code, oc, scale,
         out.data_ptr())
    return out


def embedding_grad(grad_out, tokens, vocab, scale=1.0, grad_dtype=None, out=None, workspace=None):
    """Gradient of embedding_lookup's table (vocab x dim): scale times the sum of
    grad_out over every token's rows, in a fixed order."""
    ld, tb = _rows(grad_out, "grad_out"), _int(tokens, "tokens")
    (n, dim), vocab = grad_out.shape, int(vocab)
    if tokens.numel() != n:
        _bad(f"tokens: expected {n}, one for each row of grad_out, got {tokens.numel()}")
    if not 1 <= vocab <= 1 << 26:
        _bad("the number of keys must be in [1, 2^26]")
    dev = _device(grad_out, tokens)
    grad_dtype = grad_dtype or (out.dtype if out is not None else grad_out.dtype)
    code, oc = _float(grad_out.dtype, "grad_out"), _float(grad_dtype, "out")
    out = _result(out, (vocab, dim), grad_dtype, dev, "out")
    buf, ws, nb = _scratch(workspace, dev, _workspace_bytes("mo_embedding_grad_workspace_bytes", n, vocab, dim))
    _run("mo_embedding_grad", dev, grad_out.data_ptr(), ld, tokens.data_ptr(), tb, n, vocab, dim, code, oc, scale,
         out.data_ptr(), ws, nb)
    return out


def _experts(w, offsets):
    if w.dim() != 3 or not w.is_contiguous():
        _bad("w: expected a contiguous tensor [experts][m][k]")
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or not offsets.is_contiguous():
        _bad("offsets: expected a contiguous int32 vector")
    if offsets.numel() != w.shape[0] + 1:
        _bad(f"offsets: expected {w.shape[0] + 1} values, got {offsets.numel()}")
    return w.shape


def expert_matmul(x, w, offsets, out_dtype=None, out=None):
    """y[r] = x[r] w[e]^T for the rows r of expert e, offsets[e] .. offsets[e + 1] - 1;
    zeros for rows of no expert.  x: n x k, w: experts x m x k, y: n x m."""
    ld = _rows(x, "x")
    e, m, k = _experts(w, offsets)
    n = x.shape[0]
    if x.shape[1] != k:
        _bad(f"x: expected {k} columns, as w has, got {x.shape[1]}")
    if x.dtype != w.dtype:
        raise MatoptError(-2, "x and w must share one dtype")
    dev = _device(x, w, offsets)
    out_dtype = out_dtype or (out.dtype if out is not None else x.dtype)
    code, oc = _float(x.dtype, "x"), _float(out_dtype, "out")
    out = _result(out, (n, m), out_dtype, dev, "out")
    _run("mo_expert_matmul", dev, x.data_ptr(), ld, w.data_ptr(), offsets.data_ptr(), e, n, k, m, code, oc,
         out.data_ptr())
    return out


def expert_input_grad(dy, w, offsets, out_dtype=None, out=None):
    """dx[r] = dy[r] w[e] for the rows r of expert e; zeros for rows of no expert.
    dy: n x m, w: experts x m x k, dx: n x k."""
    ld = _rows(dy, "dy")
    e, m, k = _experts(w, offsets)
    n = dy.shape[0]
    if dy.shape[1] != m:
        _bad(f"dy: expected {m} columns, as w has rows, got {dy.shape[1]}")
    if dy.dtype != w.dtype:
        raise MatoptError(-2, "dy and w must share one dtype")
    dev = _device(dy, w, offsets)
    out_dtype = out_dtype or (out.dtype if out is not None else dy.dtype)
    code, oc = _float(dy.dtype, "dy"), _float(out_dtype, "out")
    out = _result(out, (n, k), out_dtype, dev, "out")
    _run("mo_expert_input_grad", dev, dy.data_ptr(), ld, w.data_ptr(), offsets.data_ptr(), e, n, k, m, code, oc,
         out.data_ptr())
    return out


def expert_weight_grad(dy, x, offsets, out_dtype=None, out=None):
    """dw[e] = the sum of dy[r]^T x[r] over the rows r of expert e (experts x m x k): the
    gradients that the owner-local step takes, one matrix per expert."""
    ldy, ldx = _rows(dy, "dy"), _rows(x, "x")
    (n, m), k = dy.shape, x.shape[1]
    if x.shape[0] != n:
        _bad(f"x: expected {n} rows, as dy has, got {x.shape[0]}")
    if dy.dtype != x.dtype:
        raise MatoptError(-2, "dy and x must share one dtype")
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or not offsets.is_contiguous() or offsets.numel() < 2:
        _bad("offsets: expected a contiguous int32 vector of experts + 1 values")
    e = offsets.numel() - 1
    dev = _device(dy, x, offsets)
    out_dtype = out_dtype or (out.dtype if out is not None else dy.dtype)
    code, oc = _float(dy.dtype, "dy"), _float(out_dtype, "out")
    out = _result(out, (e, m, k), out_dtype, dev, "out")
    _run("mo_expert_weight_grad", dev, dy.data_ptr(), ldy, x.data_ptr(), ldx, offsets.data_ptr(), e, n, k, m, code,
         oc, out.data_ptr())
    return out


def _row_values(t, name, n):
    if t.dtype != torch.float32 or t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        _bad(f"{name}: expected a contiguous float32 vector of {n} values")


def _distill(logits, indices, teacher, temperature, lse=None, row_grad=None):
    ld, code = _rows(logits, "logits"), _float(logits.dtype, "logits")
    ib = _INT.get(indices.dtype)
    if ib is None:
        raise MatoptError(-2, f"indices: expected int32 or int64, got {indices.dtype}")
    if teacher.dtype != torch.float32:
        raise MatoptError(-2, f"teacher: expected float32, got {teacher.dtype}")
    n, v = logits.shape
    shape = indices.shape
    if len(shape) != 2 or shape[0] != n or shape != teacher.shape:
        _bad(f"indices and teacher: expected one shape [{n}][k]")
    if not indices.is_contiguous() or not teacher.is_contiguous():
        _bad("indices and teacher must be contiguous")
    if lse is not None:
        _row_values(lse, "lse", n)
    if row_grad is not None:
        _row_values(row_grad, "row_grad", n)
    if not 0.0 < temperature < float("inf"):
        _bad("temperature must be finite and > 0")
    return _device(logits, indices, teacher, lse, row_grad), ld, ib, n, v, shape[1], code


def distill_forward(logits, indices, teacher, temperature=1.0):
    """(loss, lse) per row: the divergence of the student's softmax from the teacher's,
    which is given by its top logits (indices and teacher, n x k, ids outside the
    vocabulary left out), times temperature^2."""
    dev, ld, ib, n, v, k, code = _distill(logits, indices, teacher, temperature)
    loss, lse = teacher.new_empty(n), teacher.new_empty(n)
    _run("mo_distill_forward", dev, logits.data_ptr(), ld, indices.data_ptr(), ib, teacher.data_ptr(), n, v, k, code,
         temperature, loss.data_ptr(), lse.data_ptr())
    return loss, lse


def distill_backward(logits, lse, indices, teacher, row_grad, temperature=1.0, out=None):
    """Gradient of the logits for the rows' weights row_grad, from distill_forward's lse.
    Not in place."""
    dev, ld, ib, n, v, k, code = _distill(logits, indices, teacher, temperature, lse, row_grad)
    out = _result(out, (n, v), logits.dtype, dev, "out")
    _run("mo_distill_backward", dev, logits.data_ptr(), ld, lse.data_ptr(), indices.data_ptr(), ib,
         teacher.data_ptr(), row_grad.data_ptr(), n, v, k, code, temperature, out.data_ptr(), v)
    return out


def distill_forward_backward(logits, indices, teacher, row_grad, temperature=1.0, out=None):
    """(loss, lse, gradient of the logits) in one pass, where the rows' weights are known.
    Not in place."""
    dev, ld, ib, n, v, k, code = _distill(logits, indices, teacher, temperature, None, row_grad)
    loss, lse = teacher.new_empty(n), teacher.new_empty(n)
    out = _result(out, (n, v), logits.dtype, dev, "out")
    _run("mo_distill_forward_backward", dev, logits.data_ptr(), ld, indices.data_ptr(), ib, teacher.data_ptr(),
         row_grad.data_ptr(), n, v, k, code, temperature, loss.data_ptr(), lse.data_ptr(), out.data_ptr(), v)
    return loss, lse, out
