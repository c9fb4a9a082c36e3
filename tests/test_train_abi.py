"""CPU checks of the training-block operators' C ABI and binding: exported
symbols, workspace queries, and every refusal, which comes before anything is
launched (nothing here launches a kernel)."""

import ctypes
import math
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "msign_train.h")

train = pytest.importorskip("msign_newton_schulz_amd._train")

OK, ARG, DTYPE, SHAPE, WORKSPACE, ALIAS = range(6)
INVALID = (1 << 64) - 1


def _lib():
    from msign_newton_schulz_amd import LIB_PATH
    if not os.path.exists(LIB_PATH):
        pytest.skip("libmsign.so not built")
    try:
        return train._library()
    except OSError as e:  # pragma: no cover - missing HIP runtime
        if "undefined symbol" in str(e):
            raise
        pytest.skip(f"cannot load libmsign.so here: {e}")


def test_library_exports_every_declared_symbol():
    lib = _lib()
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:const\s+)?[A-Za-z_]\w*\s*\*?\s+\*?([a-z_]\w*)\s*\(", text, flags=re.M))
    assert {"ffn_forward", "ffn_backward", "add_rms_norm", "add_rms_norm_backward", "distill_topk"} <= names
    for name in names:
        assert hasattr(lib, name), name


# addresses that no check may follow: far apart, 256-byte aligned
def at(i):
    return (i + 1) << 36


def block(tokens=8, dim=64, hidden=128, dtype=1, activation=0, **kw):
    b = train._Block(tokens, dim, hidden, dtype, activation, at(0), at(1), at(2), at(3), dim, dim, dim, hidden)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def forward(lib, b, y=at(4), ldy=None, gate=at(5), up=at(6), ld_act=None, ws=at(7), wsb=1 << 34):
    return lib.ffn_forward(b, y, ldy if ldy is not None else max(b.dim, 1), gate, up,
                           ld_act if ld_act is not None else max(b.hidden, 1), ws, wsb, None)


def backward(lib, b, dy=at(4), ld_dy=None, gate=at(5), up=at(6), dx=at(8), dwg=at(9), dwu=at(10), dwd=at(11),
             ws=at(7), wsb=1 << 34):
    return lib.ffn_backward(b, dy, ld_dy if ld_dy is not None else b.dim, gate, up, b.hidden, dx, dwg, dwu, dwd, ws,
                            wsb, None)


def test_ffn_workspace():
    lib = _lib()
    query = lib.ffn_forward_workspace_bytes
    assert query(block(tokens=0)) == 0
    assert query(block(tokens=100)) >= 100 * 128 * 2
    assert query(block(dtype=7)) == INVALID and query(block(dim=-1)) == INVALID
    assert query(block(hidden=(1 << 20) + 1)) == INVALID and query(block(tokens=(1 << 24) + 1)) == INVALID
    # an operand that starts off 16 bytes or whose pitch does is copied
    assert query(block(w_up=at(2) + 2)) >= query(block()) + 128 * 64 * 2
    assert query(block(ldx=65)) >= query(block()) + 8 * 64 * 2
    back = lib.ffn_backward_workspace_bytes
    assert back(block(), at(4), 64) >= 3 * 8 * 128 * 2
    assert back(block(), at(4) + 2, 64) > back(block(), at(4), 64)
    assert back(block(tokens=-1), at(4), 64) == INVALID


def test_ffn_refusals():
    lib = _lib()
    for run in (forward, backward):
        assert run(lib, block(dtype=3)) == DTYPE
        assert run(lib, block(tokens=-1)) == SHAPE
        assert run(lib, block(dim=(1 << 20) + 1)) == SHAPE
        assert run(lib, block(activation=2)) == ARG
        assert run(lib, block(x=0)) == ARG
        assert run(lib, block(w_down=at(3) + 1)) == ARG
        assert run(lib, block(ld_gate=63)) == ARG
        assert run(lib, block(ldx=(1 << 21) + 1)) == ARG
        assert run(lib, block(), ws=None) == WORKSPACE
        assert run(lib, block(), wsb=16) == WORKSPACE
        assert run(lib, block(), ws=at(7) + 128) == WORKSPACE
        assert run(lib, block(), ws=at(1)) == ALIAS
        assert run(lib, block(), up=None) == ARG
    assert lib.msign_train_last_error()
    assert forward(lib, block(), y=None) == ARG
    assert forward(lib, block(), ldy=63) == ARG
    assert forward(lib, block(), ld_act=127) == ARG
    assert forward(lib, block(), y=at(0)) == ALIAS
    assert forward(lib, block(), gate=at(4)) == ALIAS
    assert backward(lib, block(), dx=at(4)) == ALIAS
    assert backward(lib, block(), dwu=at(9) + 2) == ALIAS
    assert backward(lib, block(), dwd=None) == ARG
    assert backward(lib, block(), dy=at(4) + 1) == ARG
    assert forward(lib, block(tokens=0)) == OK


def norm(lib, x=at(0), ldx=64, r=at(1), ldr=64, w=at(2), y=at(3), h=at(4), rstd=at(5), tokens=8, dim=64, dtype=1,
         wdt=1, eps=1e-6):
    return lib.add_rms_norm(x, ldx, r, ldr, w, y, h, rstd, tokens, dim, dtype, wdt, eps, None)


def norm_back(lib, dy=at(0), ld_dy=64, h=at(1), ldh=64, rstd=at(2), w=at(3), dh=at(4), ld_dh=64, dx=at(5), dw=at(6),
              tokens=8, dim=64, dtype=1, wdt=1, ws=at(7), wsb=1 << 30):
    return lib.add_rms_norm_backward(dy, ld_dy, h, ldh, rstd, w, dh, ld_dh, dx, dw, tokens, dim, dtype, wdt, ws, wsb,
                                     None)


def test_norm_refusals():
    lib = _lib()
    assert norm(lib, dtype=9) == DTYPE and norm(lib, wdt=-1) == DTYPE
    assert norm(lib, dim=32769) == SHAPE and norm(lib, tokens=-1) == SHAPE
    for eps in (0.0, -1.0, math.inf, math.nan):
        assert norm(lib, eps=eps) == ARG
    assert norm(lib, ldx=63) == ARG and norm(lib, x=None) == ARG and norm(lib, h=None) == ARG
    assert norm(lib, w=at(2) + 1) == ARG and norm(lib, rstd=at(5) + 2) == ARG
    assert norm(lib, y=at(0)) == ALIAS and norm(lib, y=at(4)) == ALIAS and norm(lib, h=at(1) + 2) == ALIAS
    assert norm(lib, h=at(1), ldr=65) == ALIAS
    assert norm(lib, tokens=0, x=None) == OK
    assert norm_back(lib, dtype=9) == DTYPE and norm_back(lib, dim=40000) == SHAPE
    assert norm_back(lib, dw=None) == ARG and norm_back(lib, ld_dh=10) == ARG and norm_back(lib, rstd=None) == ARG
    assert norm_back(lib, ws=None) == WORKSPACE and norm_back(lib, wsb=8) == WORKSPACE
    assert norm_back(lib, dx=at(1)) == ALIAS and norm_back(lib, dw=at(3)) == ALIAS and norm_back(lib, ws=at(0)) == ALIAS
    assert norm_back(lib, dx=at(0), ld_dy=65) == ALIAS and norm_back(lib, dx=at(4) + 2) == ALIAS
    assert lib.add_rms_norm_backward_workspace_bytes(4, -1) == INVALID
    assert lib.add_rms_norm_backward_workspace_bytes(0, 64) == 0


def distill(lib, z=at(0), ldz=100, idx=at(1), i64=1, t=at(2), tdt=0, grad=at(3), stride=1, loss=at(4), dz=at(5), rows=6,
            vocab=100, top=4, tau=1.0, dtype=1):
    return lib.distill_topk(z, ldz, idx, i64, t, tdt, grad, stride, loss, dz, rows, vocab, top, tau, dtype, None)


def test_distill_refusals():
    lib = _lib()
    assert distill(lib, dtype=5) == DTYPE and distill(lib, tdt=5) == DTYPE
    assert distill(lib, vocab=0) == SHAPE and distill(lib, top=1025) == SHAPE and distill(lib, rows=-1) == SHAPE
    assert distill(lib, vocab=(1 << 21) + 1, ldz=1 << 22) == SHAPE
    for tau in (0.0, -1.0, math.inf, math.nan):
        assert distill(lib, tau=tau) == ARG
    assert distill(lib, ldz=99) == ARG and distill(lib, grad=None) == ARG and distill(lib, stride=-1) == ARG
    assert distill(lib, i64=2) == ARG and distill(lib, idx=at(1) + 4) == ARG and distill(lib, loss=None) == ARG
    assert distill(lib, loss=at(0)) == ALIAS and distill(lib, dz=at(0) + 2) == ALIAS
    assert distill(lib, dz=at(0), ldz=101) == ALIAS and distill(lib, dz=at(2)) == ALIAS
    assert distill(lib, rows=0, z=None) == OK


def test_binding_refuses_what_it_can_see():
    import msign_newton_schulz_amd as M
    x, w, wd = torch.zeros(4, 8), torch.zeros(16, 8), torch.zeros(8, 16)
    with pytest.raises(ValueError, match="GPU"):
        M.gated_ffn(x, w, w, wd)
    with pytest.raises(ValueError, match="activation"):
        M.gated_ffn(x, w, w, wd, activation="relu")
    with pytest.raises(ValueError, match="shapes"):
        M.gated_ffn(x, w, w, w)
    with pytest.raises(ValueError, match="dtype"):
        M.gated_ffn(x, w, w.half(), wd)
    with pytest.raises(ValueError, match="dy"):
        class OnGpu(torch.Tensor):
            is_cuda = True
        g = torch.zeros(4, 16)
        M.gated_ffn_backward(torch.zeros(3, 8), *[t.as_subclass(OnGpu) for t in (x, w, w, wd)], g, g)
    with pytest.raises(ValueError, match="weight"):
        M.add_rms_norm(x, torch.zeros(9))
    with pytest.raises(ValueError, match="residual"):
        M.add_rms_norm(x, torch.zeros(8), x.half())
    with pytest.raises(ValueError, match="rstd"):
        M.add_rms_norm_backward(x, x, torch.zeros(5), torch.zeros(8))
    idx = torch.zeros(4, 2, dtype=torch.int64)
    with pytest.raises(ValueError, match="teacher"):
        M.distill_topk(x, idx, torch.zeros(4, 3))
    with pytest.raises(TypeError, match="int32"):
        M.distill_topk(x, idx.short(), torch.zeros(4, 2))
    with pytest.raises(TypeError, match="float32"):
        M.distill_topk_grad(x, idx, torch.zeros(4, 2), torch.zeros(4).double())
    with pytest.raises(ValueError, match="grad"):
        M.distill_topk_grad(x, idx, torch.zeros(4, 2), torch.zeros(3))
    with pytest.raises(ValueError, match="out"):
        M.distill_topk_grad(x, idx, torch.zeros(4, 2), torch.zeros(4), out=torch.zeros(4, 9))


MOST_ROWS = 1 << 24


@pytest.mark.parametrize("rows", [(1 << 21) + 1, MOST_ROWS])
def test_row_operators_take_up_to_2_24_rows(rows):
    """The vectors with one element a row have no pitch to refuse: a later
    check answers."""
    lib = _lib()
    assert norm(lib, tokens=rows, y=at(0)) == ALIAS
    assert norm_back(lib, tokens=rows, ws=None) == WORKSPACE
    assert distill(lib, rows=rows, loss=at(0)) == ALIAS
    assert norm(lib, tokens=MOST_ROWS + 1) == SHAPE and distill(lib, rows=MOST_ROWS + 1) == SHAPE
    assert norm(lib, tokens=rows, rstd=None) == ARG and norm(lib, tokens=rows, rstd=at(5) + 2) == ARG
    assert norm_back(lib, tokens=rows, rstd=None) == ARG and distill(lib, rows=rows, loss=at(4) + 2) == ARG


def test_row_operators_take_any_pitch_that_memory_holds():
    """The last token's logits of every sequence, or every thousandth row, have
    pitches past the products' limit: a later check answers."""
    lib = _lib()
    far = 1 << 31
    assert norm(lib, ldx=far, y=at(0)) == ALIAS and norm(lib, ldr=far, y=at(0)) == ALIAS
    for pitch in ("ld_dy", "ldh", "ld_dh"):
        assert norm_back(lib, ws=None, **{pitch: far}) == WORKSPACE
    assert distill(lib, ldz=far, loss=at(0)) == ALIAS
    # rows that reach into an output are still seen
    assert norm(lib, ldx=far, y=at(0) + 4 * far) == ALIAS
    too_far = (1 << 36) + 1
    assert norm(lib, ldx=too_far) == ARG and norm_back(lib, ldh=too_far) == ARG and distill(lib, ldz=too_far) == ARG
    assert distill(lib, stride=too_far) == ARG


@pytest.mark.parametrize("dtype,size", [(0, 4), (1, 2), (2, 2)])
@pytest.mark.parametrize("tokens,dim,hidden", [(1, 1024, 4096), (16, 4096, 4096), (32, 512, 2048)])
def test_ffn_workspace_of_a_few_tokens_is_the_hidden_activations(tokens, dim, hidden, dtype, size):
    """The kernels for a few tokens split no tiles, so need no room for parts."""
    need = _lib().ffn_forward_workspace_bytes(block(tokens=tokens, dim=dim, hidden=hidden, dtype=dtype))
    assert need == tokens * hidden * size


def test_assembly_declares_the_registers_that_it_names():
    """m0 and the condition registers are the compiler's too: a statement that
    writes one lists it."""
    folder = os.path.join(ROOT, "msign_newton_schulz_amd", "csrc")
    seen = 0
    for name in sorted(os.listdir(folder)):
        for stmt in re.findall(r"\basm\b[^;]*;", open(os.path.join(folder, name)).read()):
            code, _, lists = stmt.partition("::") if "::" in stmt else stmt.partition(" : ")
            for reg in ("m0", "vcc", "exec"):
                if re.search(rf"\b{reg}\b", code):
                    seen += 1
                    assert f'"{reg}"' in lists, (name, stmt)
    assert seen > 0
