"""The training-step operators on the host: the struct layout the ctypes binding assumes,
the refusals of every entry point (all before anything is enqueued: no GPU here), workspace
sizes, and the FP64 statements pinned to finite differences."""

import ctypes
import os
import subprocess

import pytest
import torch

from oracle import train_ops as O

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F32, BF16 = 0, 1
OK, INVALID, ID, ALIGN, WS, UNSUP = 0, 1, 3, 4, 5, 6


@pytest.fixture(scope="module")
def abi():
    from speculative_decoding_draft_vocab_b200 import build as _build
    _build.build()
    from speculative_decoding_draft_vocab_b200 import abi as _abi
    return _abi


def test_struct_layout_matches_ctypes(abi, tmp_path):
    classes = (abi.dspark_lce_problem_t, abi.dspark_lce_out_t, abi.dspark_lce_grads_t, abi.dspark_embed_problem_t,
               abi.dspark_tensor_t)
    lines = []
    for c in classes:
        lines.append(f'printf("%zu\\n", sizeof({c.__name__}));')
        lines += [f'printf("%zu\\n", offsetof({c.__name__}, {f}));' for f, _ in c._fields_]
    src = tmp_path / "layout.c"
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"dspark.h\"\nint main(void) {\n"
                   + "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()]
    want = []
    for c in classes:
        want.append(ctypes.sizeof(c))
        want += [getattr(c, f).offset for f, _ in c._fields_]
    assert got == want


# ------------------------------------------------------------- linear cross entropy
def _lce(abi, **kw):
    p = abi.dspark_lce_problem_t()
    p.R, p.V, p.H = 16, 1000, 64
    p.hidden, p.hidden_ld = 0x10000, 64
    p.weight, p.weight_ld = 0x20000, 64
    p.targets, p.ignore_index = 0x30000, -100
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def _lce_grads(abi, **kw):
    g = abi.dspark_lce_grads_t()
    g.dhidden, g.dhidden_ld = 0x40000, 64
    g.dweight, g.dweight_ld, g.dweight_dtype = 0x50000, 64, BF16
    for k, v in kw.items():
        setattr(g, k, v)
    return g


def _lce_fwd(abi, p, ws=0x100000, n=1 << 40, out=True):
    o = abi.dspark_lce_out_t()
    return abi.dspark_lce_fwd(ctypes.byref(p) if p is not None else None, ctypes.byref(o) if out else None,
                              ctypes.c_void_p(ws), n, None)


def _lce_bwd(abi, p, g, ws=0x100000, n=1 << 40):
    return abi.dspark_lce_bwd(ctypes.byref(p), ctypes.byref(g) if g is not None else None, ctypes.c_void_p(ws), n,
                              None)


@pytest.mark.parametrize("change,status", [
    (dict(R=0), INVALID), (dict(V=0), INVALID), (dict(H=0), INVALID), (dict(R=-1), INVALID),
    (dict(hidden=0), INVALID), (dict(weight=0), INVALID), (dict(targets=0), INVALID),
    (dict(hidden_ld=56), INVALID), (dict(weight_ld=56), INVALID),
    (dict(hidden_grad_only=2), INVALID), (dict(z_alpha=-1.0), INVALID), (dict(z_alpha=float("nan")), INVALID),
    (dict(H=60), ALIGN), (dict(hidden_ld=68), ALIGN), (dict(weight_ld=68), ALIGN),
    (dict(hidden=0x10008), ALIGN), (dict(weight=0x20002), ALIGN),
    (dict(R=(1 << 24) + 1), UNSUP), (dict(V=(1 << 30) + 1), UNSUP), (dict(H=(1 << 20) + 8), UNSUP),
    (dict(R=1 << 24, V=1 << 30), UNSUP),
])
def test_lce_refuses_a_bad_problem(abi, change, status):
    assert _lce_fwd(abi, _lce(abi, **change)) == status
    assert _lce_bwd(abi, _lce(abi, **change), _lce_grads(abi)) == status


def test_lce_refuses_missing_structs_and_workspaces(abi):
    p = _lce(abi)
    assert _lce_fwd(abi, None) == INVALID
    assert _lce_fwd(abi, p, out=False) == INVALID
    assert _lce_bwd(abi, p, None) == INVALID
    assert _lce_fwd(abi, p, ws=0) == WS
    assert _lce_fwd(abi, p, ws=0x100080) == ALIGN
    need = abi.dspark_lce_workspace_size(ctypes.byref(p), None)
    assert need > 0 and _lce_fwd(abi, p, n=need - 1) == WS
    g = _lce_grads(abi)
    more = abi.dspark_lce_workspace_size(ctypes.byref(p), ctypes.byref(g))
    assert more > need and _lce_bwd(abi, p, g, n=more - 1) == WS


@pytest.mark.parametrize("change,status", [
    (dict(dhidden=0, dweight=0), INVALID), (dict(dhidden_ld=56), INVALID), (dict(dweight_ld=56), INVALID),
    (dict(dweight_dtype=2), INVALID), (dict(accumulate=1), UNSUP),
    (dict(dhidden=0x40008), ALIGN), (dict(dhidden_ld=68), ALIGN), (dict(dweight=0x50004), ALIGN),
    (dict(dweight_ld=68), ALIGN), (dict(dweight_dtype=F32, dweight_ld=66), ALIGN),
])
def test_lce_refuses_bad_gradients(abi, change, status):
    assert _lce_bwd(abi, _lce(abi), _lce_grads(abi, **change)) == status


def test_lce_hidden_grad_only(abi):
    """No head gradient may be asked for, and at a large vocabulary the forward needs the
    backward's workspace."""
    assert _lce_bwd(abi, _lce(abi, hidden_grad_only=1), _lce_grads(abi)) == INVALID
    size = lambda p, g=None: abi.dspark_lce_workspace_size(  # noqa: E731
        ctypes.byref(p), ctypes.byref(g) if g is not None else None)
    only = _lce_grads(abi, dweight=0)
    small, large = _lce(abi, hidden_grad_only=1), _lce(abi, V=20000, hidden_grad_only=1)
    assert size(small) < size(small, only)
    assert size(large) == size(large, only) > size(_lce(abi, V=20000))
    assert _lce_fwd(abi, large, n=size(large) - 1) == WS


def test_lce_workspace_is_far_below_the_logits(abi):
    p = _lce(abi, R=8192, V=151936, H=4096)
    fwd = abi.dspark_lce_workspace_size(ctypes.byref(p), None)
    bwd = abi.dspark_lce_workspace_size(ctypes.byref(p), ctypes.byref(_lce_grads(abi)))
    logits = 2 * p.R * p.V
    assert fwd < logits // 16
    assert bwd < fwd + (256 << 20) + 5 * p.R * p.H  # the piece of dz, one FP32 plane
    # the FP32 logits stay where they take at most 320 MiB, and only beside a backward
    q = _lce(abi, R=448, V=151936, H=64)
    assert abi.dspark_lce_workspace_size(ctypes.byref(q), None) < 16 << 20
    kept = abi.dspark_lce_workspace_size(ctypes.byref(q), ctypes.byref(_lce_grads(abi)))
    q.R = 600
    assert 6 * 448 * q.V < kept < 7 * 448 * q.V
    assert abi.dspark_lce_workspace_size(ctypes.byref(q), ctypes.byref(_lce_grads(abi))) < 3 * 600 * q.V
    frozen = abi.dspark_lce_workspace_size(ctypes.byref(p), ctypes.byref(_lce_grads(abi, dhidden=0)))
    assert frozen <= bwd - 4 * p.R * p.H
    assert abi.dspark_lce_workspace_size(None, None) == 0
    assert abi.dspark_lce_workspace_size(ctypes.byref(_lce(abi, R=0)), None) == 0


# ----------------------------------------------------------------------- embedding
def _emb(abi, **kw):
    p = abi.dspark_embed_problem_t()
    p.R, p.Vt, p.D, p.dtype, p.ids, p.scale = 16, 100, 64, BF16, 0x30000, 1.0
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def _emb_fwd(abi, p, table=0x10000, tld=64, out=0x20000, old=64, ws=0x100000, n=1 << 40):
    return abi.dspark_embed_fwd(ctypes.byref(p) if p is not None else None, table, tld, out, old, ws, n, None)


def _emb_bwd(abi, p, dout=0x10000, dld=64, dt=0x20000, tld=64, dtype=F32, acc=0, ws=0x100000, n=1 << 40):
    return abi.dspark_embed_bwd(ctypes.byref(p) if p is not None else None, dout, dld, dt, tld, dtype, acc, ws, n,
                                None)


@pytest.mark.parametrize("change,status", [
    (dict(R=0), INVALID), (dict(Vt=0), INVALID), (dict(D=0), INVALID), (dict(dtype=2), INVALID),
    (dict(ids=0), INVALID), (dict(R=(1 << 24) + 1), UNSUP), (dict(Vt=(1 << 30) + 1), UNSUP),
    (dict(D=(1 << 20) + 8), UNSUP), (dict(D=60), ALIGN), (dict(D=72), INVALID),
])
def test_embed_refuses_a_bad_problem(abi, change, status):
    p = _emb(abi, **change)
    assert _emb_fwd(abi, p) == status
    assert _emb_bwd(abi, p) == status


def test_embed_refuses_bad_matrices_and_workspaces(abi):
    p = _emb(abi)
    assert _emb_fwd(abi, None) == INVALID and _emb_bwd(abi, None) == INVALID
    assert _emb_fwd(abi, p, table=0) == INVALID and _emb_fwd(abi, p, out=0) == INVALID
    assert _emb_fwd(abi, p, tld=56) == INVALID and _emb_fwd(abi, p, old=56) == INVALID
    assert _emb_fwd(abi, p, table=0x10008) == ALIGN and _emb_fwd(abi, p, old=68) == ALIGN
    assert _emb_bwd(abi, p, dtype=2) == INVALID and _emb_bwd(abi, p, dtype=BF16, acc=1) == UNSUP
    assert _emb_bwd(abi, p, dout=0) == INVALID and _emb_bwd(abi, p, dt=0) == INVALID
    assert _emb_bwd(abi, p, dt=0x20008) == ALIGN and _emb_bwd(abi, p, tld=66) == ALIGN
    for fn, grads in ((_emb_fwd, 0), (_emb_bwd, 1)):
        need = abi.dspark_embed_workspace_size(ctypes.byref(p), grads)
        assert fn(abi, p, ws=0) == WS and fn(abi, p, ws=0x100010) == ALIGN and fn(abi, p, n=need - 1) == WS
    assert abi.dspark_embed_workspace_size(None, 0) == 0


# ------------------------------------------------------------------------ clipping
def _tensors(abi, *rows):
    arr = (abi.dspark_tensor_t * len(rows))()
    for i, r in enumerate(rows):
        arr[i] = abi.dspark_tensor_t(*r)
    return arr


def _clip(abi, t, count=1, max_norm=1.0, ws=0x100000, n=1 << 40):
    return abi.dspark_grad_clip(t, count, max_norm, None, None, ws, n, None)


def test_clip_refuses(abi):
    good = _tensors(abi, (0x10000, 0x10000, 10, F32))
    assert _clip(abi, None) == INVALID and _clip(abi, good, count=0) == INVALID
    assert _clip(abi, good, count=(1 << 20) + 1) == UNSUP
    for bad in (0.0, -1.0, float("nan")):
        assert _clip(abi, good, max_norm=bad) == INVALID
    assert _clip(abi, good, ws=0) == WS and _clip(abi, good, ws=0x100001) == ALIGN
    assert _clip(abi, good, n=abi.dspark_grad_workspace_size(1) - 1) == WS
    for row, status in (((0x10000, 0x10000, -1, F32), INVALID), ((0x10000, 0x10000, 1, 2), INVALID),
                        ((0, 0x10000, 1, F32), INVALID), ((0x10000, 0, 1, F32), INVALID),
                        ((0x10002, 0x10000, 1, F32), ALIGN), ((0x10000, 0x10001, 1, BF16), ALIGN),
                        ((0x10000, 0x10000, (1 << 40) + 1, F32), UNSUP)):
        assert _clip(abi, _tensors(abi, row)) == status, row
    assert abi.dspark_grad_sumsq(good, 1, None, 0x100000, 1 << 40, None) == INVALID
    assert abi.dspark_grad_scale(good, 1, None, 1.0, None, None, 0x100000, 1 << 40, None) == INVALID
    assert abi.dspark_grad_workspace_size(0) == 0 and abi.dspark_grad_workspace_size((1 << 20) + 1) == 0


def test_python_wrappers_refuse_host_tensors():
    from speculative_decoding_draft_vocab_b200 import torch_api as T
    h, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(5, 8, dtype=torch.bfloat16)
    ids = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        T.LinearCE(h, w, ids)
    with pytest.raises(ValueError, match="CUDA"):
        T.Embedding(ids, w)
    with pytest.raises(ValueError, match="CUDA"):
        T.EmbeddingGrad(ids, h, 5)
    with pytest.raises(ValueError, match="CUDA"):
        T.GradClip([h], 1.0)
    with pytest.raises(ValueError, match="at least one"):
        T.GradClip([], 1.0)


# ------------------------------------------------- the FP64 statements' own gradients
def test_linear_ce_statement_against_differences():
    g = torch.Generator().manual_seed(5)
    h, w = torch.randn(5, 6, generator=g).double(), torch.randn(11, 6, generator=g).double()
    t = torch.tensor([3, -100, 10, 0, 3])
    a = torch.rand(5, generator=g).double()

    def loss(h, w):
        return O.linear_ce(h, w, t, a, z_alpha=0.01)["loss_num"]
    ref = O.linear_ce(h, w, t, a, z_alpha=0.01, grad_scale=1.0)
    eps = 1e-5  # central differences: error O(eps^2) of O(1) third derivatives, and 1e-16 / eps
    for x, key in ((h, "dhidden"), (w, "dweight")):
        for i in range(x.shape[0]):
            for j in range(x.shape[1]):
                old = float(x[i, j])
                x[i, j] = old + eps
                up = float(loss(h, w))
                x[i, j] = old - eps
                down = float(loss(h, w))
                x[i, j] = old
                assert abs((up - down) / (2 * eps) - float(ref[key][i, j])) < 1e-8
    assert float(ref["dhidden"][1].abs().max()) == 0.0 and ref["num_tokens"] == 4


def test_embedding_statement_against_differences():
    g = torch.Generator().manual_seed(6)
    table = torch.randn(7, 4, generator=g).double()
    ids, valid = torch.tensor([2, 2, 6, 0, 2]), torch.tensor([1, 0, 1, 1, 1], dtype=torch.uint8)
    dout = torch.randn(5, 4, generator=g).double()
    grad = O.embed_grad(ids, dout, 7, scale=1.5, valid=valid)[0]
    for i in range(7):
        for j in range(4):
            e = torch.zeros_like(table)
            e[i, j] = 1.0  # the lookup is linear: a difference of one is exact
            d = (O.embed(ids, table + e, 1.5, valid) - O.embed(ids, table, 1.5, valid)) * dout
            assert abs(float(d.sum()) - float(grad[i, j])) < 1e-12
