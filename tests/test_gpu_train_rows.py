"""The row operators of the training block (norm and distillation) where an
output takes an input's place, over more rows than workgroups, and at the
limits of row counts and pitches.

Tolerances are those of test_gpu_train.py.  An operator in place is compared
bit by bit with the same call out of place: it does the same arithmetic.
"""

import pytest
import torch

import train_reference as R
from gpu_util import announce, require_gpu
from test_gpu_train import DT, U, normal, row_tol

pytestmark = pytest.mark.gpu


def c_call(fn, t, *args):
    """fn of the C ABI on t's device and its current stream; tensors are passed
    by address."""
    from msign_newton_schulz_amd import _train
    args = [a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args]
    _train._launch(t.device, getattr(_train._library(), fn), *args)


DTYPE = {"f32": 0, "bf16": 1, "f16": 2}

# Each configuration of both passes (by the 16-byte chunks of a row), at widths
# whose chunks do not fill its threads, and full ones.
WIDTHS = [("bf16", 2000, 96), ("bf16", 5000, 500), ("bf16", 2000, 1000), ("f16", 1100, 2003), ("bf16", 1100, 4001),
          ("bf16", 800, 6001), ("f16", 800, 8100), ("bf16", 300, 16001), ("bf16", 300, 16392), ("bf16", 300, 17001),
          ("bf16", 300, 20000), ("f16", 300, 24000), ("bf16", 5, 32768), ("f32", 5000, 250), ("f32", 2000, 500),
          ("f32", 1100, 2001), ("f32", 800, 3001), ("f32", 800, 4001), ("f32", 300, 8001), ("f32", 300, 8196),
          ("f32", 300, 9001), ("f32", 300, 12288), ("f32", 300, 20001), ("f32", 5, 32768)]


@pytest.mark.parametrize("kind,rows,dim", WIDTHS)
def test_norm_backward_in_place(kind, rows, dim):
    """dx in the place of dy, of dh, and of both where they are one tensor."""
    M = require_gpu()
    dy, dh, h = (normal((rows, dim), 1.0, kind, 1 + i) for i in range(3))
    w = normal((dim,), 0.2, kind, 4) + 1
    rstd = (h.double().square().mean(1) + 1e-6).rsqrt().float()
    ws = torch.empty(768 * dim * 4 + 256, dtype=torch.uint8, device="cuda")

    def run(dy, dh, dx):
        dw = torch.empty_like(w)
        c_call("add_rms_norm_backward", h, dy, dim, h, dim, rstd, w, dh, dim, dx, dw, rows, dim, DTYPE[kind],
               DTYPE[kind], ws, ws.numel())
        return dw

    announce(f"norm backward in place {rows} {dim} {kind}")
    want = M.add_rms_norm_backward(dy, h, rstd, w, dh=dh)
    for place in ("dy", "dh"):
        a, b = dy.clone(), dh.clone()
        dx = a if place == "dy" else b
        dw = run(a, b, dx)
        torch.cuda.synchronize()
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1]), place
    want = M.add_rms_norm_backward(dy, h, rstd, w, dh=dy)
    dx = dy.clone()
    dw = run(dx, dx, dx)
    torch.cuda.synchronize()
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])


@pytest.mark.parametrize("kind,rows,dim", WIDTHS)
def test_norm_forward_in_place(kind, rows, dim):
    """h_out in the place of x, of the residual, and of both where they are one
    tensor."""
    M = require_gpu()
    x, r = normal((rows, dim), 1.0, kind, 5), normal((rows, dim), 2.0, kind, 6)
    w = normal((dim,), 0.2, kind, 7) + 1

    def run(x, r, h):
        y, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")
        c_call("add_rms_norm", x, x, dim, r, dim, w, y, h, rstd, rows, dim, DTYPE[kind], DTYPE[kind], 1e-6)
        return y, h, rstd

    announce(f"norm forward in place {rows} {dim} {kind}")
    want = M.add_rms_norm(x, w, r)
    for place in ("x", "residual"):
        a, b = x.clone(), r.clone()
        got = run(a, b, a if place == "x" else b)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), place
    want = M.add_rms_norm(x, w, x)
    a = x.clone()
    got = run(a, a, a)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_more_rows_than_a_pitch_may_have_elements():
    """Per-head norms and token-wise losses of short rows reach row counts past
    2^21.  Compared on the GPU in 64 bits."""
    M = require_gpu()
    rows, dim = (1 << 21) + 5, 24
    announce(f"norm {rows} x {dim}")
    x, r, dy = (normal((rows, dim), 1.0, "bf16", 11 + i) for i in range(3))
    w = normal((dim,), 0.2, "bf16", 14) + 1
    y, h, rstd = M.add_rms_norm(x, w, r)
    ry, rh, rs = R.rms(x.double(), r.double(), w.double(), 1e-6)
    for got, want, tol in ((y, ry, row_tol("bf16")), (h, rh, row_tol("bf16")), (rstd, rs, 40 * U["f32"])):
        assert float((got.double() - want).norm() / want.norm()) <= tol
        assert float((got.double() - want).abs().max()) <= 60 * tol * float(want.square().mean().sqrt())
    announce(f"norm backward {rows} x {dim}")
    dx, dw = M.add_rms_norm_backward(dy, h, rstd, w)
    rx, rw = R.rms_backward(dy.double(), h.double(), rstd.double(), w.double(), None)
    assert float((dx.double() - rx).norm() / rx.norm()) <= row_tol("bf16")
    assert float((dw.double() - rw).norm() / rw.norm()) <= row_tol("bf16")
    del y, ry, rh, dx, rx
    announce(f"distillation {rows} x {dim}")
    idx = (torch.arange(rows, device="cuda") * 7 % dim)[:, None]
    teacher = torch.zeros((rows, 1), device="cuda")
    loss, dz = M.distill_topk_grad(x, idx, teacher, torch.tensor(1.0, device="cuda"))
    logq = x.double().log_softmax(1)
    assert float((loss.double() + logq.gather(1, idx)[:, 0]).abs().max()) <= 40 * U["f32"] * 12
    want = logq.exp().scatter_add_(1, idx, torch.full_like(idx, -1, dtype=torch.float64))
    assert float((dz.double() - want).norm() / want.norm()) <= row_tol("bf16")


def test_row_operators_with_pitches_past_2_21():
    """The last token's logits of each sequence and every n-th token's row."""
    M = require_gpu()
    announce("distillation of last tokens")
    batch, length, vocab = 5, 41, 65539
    logits = normal((batch, length, vocab), 2.0, "bf16", 21)
    last = logits[:, -1]
    assert last.stride(0) > 1 << 21
    idx = torch.arange(batch * 3, device="cuda").view(batch, 3) * 4001
    teacher = normal((batch, 3), 1.0, "f32", 22)
    grad = torch.ones(batch, device="cuda")
    got = M.distill_topk_grad(last, idx, teacher, grad)
    want = M.distill_topk_grad(last.contiguous(), idx, teacher, grad)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(M.distill_topk(last, idx, teacher), want[0])
    announce("norm of every 8193rd token")
    wide = normal((4 * 8193, 257), 1.0, "bf16", 23)
    x, r = wide[::8193], wide[1::8193]
    assert x.stride(0) > 1 << 21
    w = normal((257,), 0.2, "bf16", 24) + 1
    y, h, rstd = M.add_rms_norm(x, w, r)
    want = M.add_rms_norm(x.contiguous(), w, r.contiguous())
    assert all(torch.equal(a, b) for a, b in zip((y, h, rstd), want))
    got = M.add_rms_norm_backward(r, x, rstd, w, dh=wide[2::8193])
    want = M.add_rms_norm_backward(r.contiguous(), x.contiguous(), rstd, w, dh=wide[2::8193].contiguous())
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("tau", [1e-42, 1e-39, 1e-37, 1e-20])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_distill_at_tiny_temperatures(kind, tau):
    """Below 2^-128 log2(e) the reciprocal of tau is past fp32's range; the
    softmax is then one at the largest logit.  With p and q there, loss =
    tau sum_k p_k (t_k - t_max - z_k + z_max) up to tau^2 log terms, and the
    gradient is tau grad (q - p), both exact up to fp32's rounding and, for
    the smallest, its last place 2^-149."""
    M = require_gpu()
    announce(f"distill tau {tau} {kind}")
    for vocab in (50, 5000, 170001):
        z = normal((3, vocab), 2.0, kind, 31)
        idx = torch.tensor([[1, 7, 20], [3, 4, 5], [0, 30, 49]], device="cuda")
        teacher = torch.tensor([[2.0, 1.0, 0.0], [0.0, 3.0, 1.0], [1.0, 0.0, 2.0]], device="cuda")
        z[0, 1] = 40.0  # the student agrees
        z[1, 9] = 40.0  # it does not
        z[2, 49] = 40.0
        grad = torch.tensor([1.0, 1.0, 0.5], device="cuda")
        loss, dz = M.distill_topk_grad(z, idx, teacher, grad, temperature=tau)
        only = M.distill_topk(z, idx, teacher, temperature=tau)
        want = tau * torch.tensor([0.0, 40.0 - float(z[1, 4]), 0.0], dtype=torch.float64, device="cuda")
        slack = 1e-5 * tau + 2.0 ** -149
        assert float((loss.double() - want).abs().max()) <= 100 * slack
        assert torch.equal(loss, only)
        full = torch.zeros((3, vocab), dtype=torch.float64, device="cuda")
        full[1, 9], full[1, 4] = tau, -tau
        # (bf16 holds the gradient itself to 2^-8, and to 2^-133 below its normal range)
        assert float((dz.double() - full).abs().max()) <= (2.0 ** -8 * tau + 2.0 ** -133 if kind == "bf16" else slack)


def close(got, want, tol):
    """Relative in the 2-norm and, for every element, in multiples of the mean
    size."""
    d = (got.double() - want).abs()
    assert float(d.norm()) <= tol * float(want.norm())
    assert float(d.max()) <= 60 * tol * float(want.square().mean().sqrt())


# More rows than resident workgroups (4096 of 64 threads, 768 or 1024 of 256,
# 512 of 512, 256 of 1024), in every configuration of the forward pass.
@pytest.mark.parametrize("kind,rows,dim", [("bf16", 5000, 96), ("f16", 4500, 1000), ("bf16", 1500, 2003),
                                           ("bf16", 900, 4099), ("f16", 600, 8200), ("bf16", 300, 12001),
                                           ("bf16", 300, 30001), ("f32", 5000, 95), ("f32", 900, 2051),
                                           ("f32", 300, 20001)])
@pytest.mark.parametrize("with_residual", [True, False])
def test_norm_walks_over_rows(kind, rows, dim, with_residual):
    """Every row, compared on the GPU in 64 bits."""
    M = require_gpu()
    announce(f"norm walk {rows} {dim} {kind} {with_residual}")
    x = normal((rows, dim), 1.0, kind, 41)
    x *= (1 + torch.arange(rows, device="cuda") % 7)[:, None].to(x.dtype)  # (neighbouring rows have other norms)
    r = normal((rows, dim), 1.0, kind, 42) if with_residual else None
    w = normal((dim,), 0.2, kind, 43) + 1
    y, h, rstd = M.add_rms_norm(x, w, r)
    ry, rh, rs = R.rms(x.double(), None if r is None else r.double(), w.double(), 1e-6)
    close(y, ry, row_tol(kind))
    close(rstd, rs, 40 * U["f32"])
    if with_residual:
        close(h, rh, row_tol(kind))


def test_norm_backward_walks_over_rows_of_one_wave():
    """Four rows a workgroup and more of them than 768 workgroups take at once."""
    M = require_gpu()
    for kind, rows, dim in (("bf16", 4001, 96), ("f32", 7003, 251), ("f16", 3500, 1000)):
        announce(f"norm backward walk {rows} {dim} {kind}")
        dy, h, dh = (normal((rows, dim), 1.0, kind, 51 + i) for i in range(3))
        w = normal((dim,), 0.2, kind, 55) + 1
        rstd = (h.double().square().mean(1) + 1e-6).rsqrt().float()
        dx, dw = M.add_rms_norm_backward(dy, h, rstd, w, dh=dh)
        rx, rw = R.rms_backward(dy.double(), h.double(), rstd.double(), w.double(), dh.double())
        close(dx, rx, row_tol(kind))
        # (f32: sums over the rows, as a product's)
        close(dw, rw, 100 * U["f32"] if kind == "f32" else row_tol(kind))


# Resident workgroups: 3072 of 64 threads, 1792 (loss), 1280, 1024 or 768 of
# 256, 512 or 256 of 512, 256 of 1024.
@pytest.mark.parametrize("kind,rows,vocab", [("bf16", 1500, 5), ("bf16", 4000, 130), ("f16", 3500, 3001), ("bf16", 1500, 6001),
                                             ("bf16", 1500, 12001), ("f16", 900, 30001), ("bf16", 600, 60001),
                                             ("bf16", 300, 90001), ("bf16", 300, 170003), ("bf16", 300, 40001),
                                             ("f32", 4000, 70), ("f32", 1500, 3003), ("f32", 900, 15001),
                                             ("f32", 300, 85001)])
def test_distill_walks_over_rows(kind, rows, vocab):
    """Loss alone and with the gradient, every row, compared on the GPU in 64
    bits."""
    M = require_gpu()
    announce(f"distill walk {rows} {vocab} {kind}")
    tau, top = 1.5, 4
    z = normal((rows, vocab), 1.0, kind, 61)
    z *= (1 + torch.arange(rows, device="cuda") % 3)[:, None].to(z.dtype)
    g = torch.Generator().manual_seed(62)
    idx = torch.randint(0, vocab, (rows, top), generator=g).cuda()
    teacher = normal((rows, top), 2.0, "f32", 63)
    grad = (torch.rand(rows, generator=g) + 0.5).cuda()
    loss, dz = M.distill_topk_grad(z, idx, teacher, grad, temperature=tau)
    only = M.distill_topk(z, idx, teacher, temperature=tau)
    logp, logq = (teacher.double() / tau).log_softmax(1), (z.double() / tau).log_softmax(1)
    want = tau * tau * (logp.exp() * (logp - logq.gather(1, idx))).sum(1)
    # (a difference of logarithms up to log(vocab) <= 12.1 and of scores)
    size = tau * tau * (12.1 + float(z.abs().max()) / tau)
    for got in (loss, only):
        assert float((got.double() - want).abs().max()) <= 40 * U["f32"] * size
    full = logq.exp_().scatter_add_(1, idx, -logp.exp()).mul_((tau * grad.double())[:, None])
    # (f16 gradients fall below its normal range: their rounding is absolute there)
    close_norm = row_tol(kind) * float(full.norm()) + (2.0 ** -25 * full.numel() ** 0.5 if kind == "f16"
                                                       else 40 * U["f32"] * tau * float(grad.norm()))
    assert float((dz.double() - full).norm()) <= close_norm
    per_row = (dz.double() - full).norm(dim=1) - 3 * row_tol(kind) * full.norm(dim=1)
    assert float(per_row.max()) <= (2.0 ** -25 * vocab ** 0.5 if kind == "f16" else 40 * U["f32"] * tau * 1.5)
