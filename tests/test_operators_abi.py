"""Refusals of the operators around the layer, on the host: no CUDA call is made
by anything tested here (the addresses are fake and never dereferenced)."""
import ctypes
import math

import pytest
import torch

import operator_reference as ref
from sparse_moe_layer_06_b200 import build, moe

A = 1 << 20  # 16-byte aligned
BF = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    build.build()
    return moe.load_library()


@pytest.fixture(autouse=True)
def launches_nothing(lib):
    before = moe.moe_launch_count()
    yield
    assert moe.moe_launch_count() == before


def problem(**kw):
    base = dict(T=64, H=256, E=16, I=128, top_k=2, num_shared=1, routed_scale=2.827,
                clip_limit=10.0, dtype=BF)
    base.update(kw)
    return moe.MoEProblem(**base)


def P(x):
    return ctypes.c_void_p(x) if x else None


def R(p):
    return ctypes.byref(p.c())


def norm(lib, p=None, x=A, res=A, w=A, eps=1e-6, ro=2 * A, y=A, q=A, s=A):
    return lib.moe_add_rmsnorm(R(p or problem()), P(x), P(res), P(w), eps, P(ro), P(y), P(q), P(s),
                               None)


def test_norm_refusals(lib):
    bad = moe.MOE_ERR_INVALID_ARG
    assert norm(lib, x=0) == bad and norm(lib, w=0) == bad
    assert norm(lib, y=0, q=0, s=0) == bad                    # nothing to write
    assert norm(lib, q=0) == bad and norm(lib, s=0) == bad    # codes without scales
    assert norm(lib, ro=A) == bad                             # both outputs in one buffer
    for name in ("x", "res", "w", "ro", "y", "q"):
        assert norm(lib, **{name: A + 8}) == bad, name
    for eps in (-1e-6, math.nan, math.inf):
        assert norm(lib, eps=eps) == bad
    assert norm(lib, p=problem(H=16448)) == moe.MOE_ERR_UNSUPPORTED
    assert norm(lib, p=problem(H=100)) == moe.MOE_ERR_UNSUPPORTED
    assert norm(lib, p=problem(T=-1)) == bad
    assert norm(lib, p=problem(T=0)) == moe.MOE_OK


def test_norm_backward_refusals(lib):
    p = problem()
    need = moe.moe_workspace_size(p, moe.MOE_CALL_ADD_RMSNORM_BACKWARD)
    assert need >= 256 + 64 * 256 * 4
    assert moe.moe_workspace_size(problem(H=16448), moe.MOE_CALL_ADD_RMSNORM_BACKWARD) == 0
    good = dict(dy=A, dres=A, h=A, w=A, dx=A, dw=A, ws=A)

    def call(n=need, eps=1e-6, pr=p, **kw):
        a = {**good, **kw}
        return lib.moe_add_rmsnorm_backward(R(pr), P(a["dy"]), P(a["dres"]), P(a["h"]), P(a["w"]),
                                            eps, P(a["dx"]), P(a["dw"]), P(a["ws"]), n, None)

    for name in ("dy", "h", "w", "dx", "dw", "ws"):
        assert call(**{name: 0}) == moe.MOE_ERR_INVALID_ARG, name
    for name in ("dy", "dres", "h", "w", "dx", "ws"):
        assert call(**{name: A + 4}) == moe.MOE_ERR_INVALID_ARG, name
    assert call(n=need - 1) == moe.MOE_ERR_WORKSPACE
    assert call(eps=math.nan) == moe.MOE_ERR_INVALID_ARG
    assert call(pr=problem(H=16448)) == moe.MOE_ERR_UNSUPPORTED


def test_balance_loss_refusals(lib):
    p = problem()
    need = moe.moe_balance_loss_workspace_size(p, 5)
    assert need > moe.moe_balance_loss_workspace_size(p, 1) == moe.moe_workspace_size(
        p, moe.MOE_CALL_BALANCE_LOSS) > 0
    assert moe.moe_balance_loss_workspace_size(p, 0) == 0
    assert moe.moe_balance_loss_workspace_size(p, (1 << 20) + 1) == 0
    assert moe.moe_balance_loss_workspace_size(problem(E=257), 1) == 0
    good = dict(logits=A, bias=A, idx=A, mask=A, off=A, loss=A, counts=A, tokens=A, prob=A, ws=A)

    def call(n_seq=5, n=need, **kw):
        a = {k: P(v) for k, v in {**good, **kw}.items()}
        return lib.moe_balance_loss(R(p), a["logits"], a["bias"], a["idx"], a["mask"], a["off"],
                                    n_seq, a["loss"], a["counts"], a["tokens"], a["prob"], a["ws"],
                                    n, None)

    for name in ("logits", "idx", "loss", "counts", "tokens", "prob", "ws"):
        assert call(**{name: 0}) == moe.MOE_ERR_INVALID_ARG, name
    assert call(off=0) == moe.MOE_ERR_INVALID_ARG          # five sequences without offsets
    assert call(n_seq=0) == moe.MOE_ERR_INVALID_ARG
    assert call(n_seq=(1 << 20) + 1) == moe.MOE_ERR_UNSUPPORTED
    assert call(n=need - 1) == moe.MOE_ERR_WORKSPACE

    def back(n_seq=5, **kw):
        a = {k: P(v) for k, v in {**dict(logits=A, off=A, counts=A, tokens=A, grad=A, dl=2 * A),
                                  **kw}.items()}
        return lib.moe_balance_loss_backward(R(p), a["logits"], None, None, a["off"], n_seq,
                                             a["counts"], a["tokens"], a["grad"], a["dl"], None)

    for name in ("logits", "off", "counts", "tokens", "grad", "dl"):
        assert back(**{name: 0}) == moe.MOE_ERR_INVALID_ARG, name
    assert back(n_seq=-1) == moe.MOE_ERR_INVALID_ARG
    assert back(dl=A) == moe.MOE_ERR_INVALID_ARG           # the logits are still read


def test_w4_refusals(lib):
    p = problem()
    need = moe.moe_workspace_size(p, moe.MOE_CALL_EXPERTS_W4)
    need_f = moe.moe_workspace_size(p, moe.MOE_CALL_FORWARD_W4)
    assert 0 < need < need_f
    for bad in (problem(H=192), problem(I=192), problem(dtype=torch.float32), problem(E=300)):
        assert moe.moe_workspace_size(bad, moe.MOE_CALL_EXPERTS_W4) == 0
    good = dict(x=A, gate=A, idx=A, w=A, q=A, s=A, sq=A, ss=A, out=A, ws=A)

    def experts(pr=p, group=128, n=need, **kw):
        a = {k: P(v) for k, v in {**good, **kw}.items()}
        return lib.moe_experts_w4(R(pr), group, a["x"], a["idx"], a["w"], a["q"], a["s"], a["sq"],
                                  a["ss"], a["out"], a["ws"], n, None)

    def forward(pr=p, group=128, n=need_f, **kw):
        a = {k: P(v) for k, v in {**good, **kw}.items()}
        return lib.moe_forward_w4(R(pr), group, a["x"], a["gate"], None, a["q"], a["s"], a["sq"],
                                  a["ss"], a["out"], None, None, a["ws"], n, None)

    for call, names in ((experts, ("x", "idx", "w", "q", "s", "sq", "ss", "out", "ws")),
                        (forward, ("x", "gate", "q", "s", "sq", "ss", "out", "ws"))):
        for name in names:
            assert call(**{name: 0}) == moe.MOE_ERR_INVALID_ARG, name
        for name in ("x", "q", "s", "sq", "ss", "out", "ws"):
            assert call(**{name: A + 8}) == moe.MOE_ERR_INVALID_ARG, name
        for name in ("q", "sq"):
            assert call(**{name: A + 16}) == moe.MOE_ERR_INVALID_ARG, name
        for group in (0, 16, 96, 256, -128):
            assert call(group=group) == moe.MOE_ERR_UNSUPPORTED
        assert call(pr=problem(H=192)) == moe.MOE_ERR_UNSUPPORTED
        assert call(pr=problem(dtype=torch.float32)) == moe.MOE_ERR_UNSUPPORTED
        assert call(pr=problem(T=0)) == moe.MOE_OK
    assert experts(n=need - 1) == moe.MOE_ERR_WORKSPACE
    assert forward(n=need_f - 1) == moe.MOE_ERR_WORKSPACE

    def enc(pr=p, group=64, n=2, w=A, q=A, s=A):
        return lib.moe_quantize_weights_w4(R(pr), group, n, P(w), P(q), P(s), None)

    for kw in (dict(w=0), dict(q=0), dict(s=0), dict(w=A + 2), dict(q=A + 8), dict(n=0),
               dict(n=65536)):
        assert enc(**kw) == moe.MOE_ERR_INVALID_ARG, kw
    assert enc(group=48) == moe.MOE_ERR_UNSUPPORTED
    assert enc(pr=problem(I=192)) == moe.MOE_ERR_UNSUPPORTED


def test_fp8_encoded_refusals(lib):
    p = problem(I=256)
    n = moe.moe_workspace_size(p, moe.MOE_CALL_FORWARD_FP8)

    def call(x=A, xq=A, xs=A, nb=n):
        return lib.moe_forward_fp8_encoded(R(p), P(x), P(xq), P(xs), P(A), None, P(A), P(A), P(A),
                                           P(A), P(A), P(A), P(A), None, None, P(A), nb, None)

    for kw in (dict(x=0), dict(xq=0), dict(xs=0), dict(xq=A + 8)):
        assert call(**kw) == moe.MOE_ERR_INVALID_ARG, kw
    assert call(nb=n - 1) == moe.MOE_ERR_WORKSPACE


def test_binding_refuses_short_wrong_and_host_tensors(lib):
    p = problem(T=8, H=128, E=4, I=128, top_k=2, num_shared=0)
    x, w = torch.zeros(8, 128, dtype=BF), torch.zeros(128, dtype=BF)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="elements"):
        moe.moe_add_rmsnorm(p, x, x[:7], w, 1e-6, None, x)
    with pytest.raises(TypeError, match="weight"):
        moe.moe_add_rmsnorm(p, x, None, w.float(), 1e-6, None, x)
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_add_rmsnorm(p, x.T.contiguous().T, None, w, 1e-6, None, x)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_add_rmsnorm(p, x, None, w, 1e-6, None, x)
    with pytest.raises(ValueError, match="required"):
        moe.moe_add_rmsnorm_backward(p, x, None, None, w, 1e-6, x, torch.zeros(128), ws)
    logits, idx = torch.zeros(8, 4), torch.zeros(8, 2, dtype=torch.int32)
    one, cnt, tok = torch.zeros(1), torch.zeros(2, 4, dtype=torch.int32), torch.zeros(
        3, dtype=torch.int32)
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError, match="token_mask"):
        moe.moe_balance_loss(p, logits, None, idx, torch.ones(8, dtype=torch.bool), off, one, cnt,
                             tok, torch.zeros(2, 4), ws)
    with pytest.raises(ValueError, match="mean_prob has 4 elements"):
        moe.moe_balance_loss(p, logits, None, idx, None, off, one, cnt, tok, torch.zeros(1, 4), ws)
    with pytest.raises(ValueError, match="offsets"):
        moe.moe_balance_loss_backward(p, logits, None, None, off.view(1, 3), cnt, tok, one, logits)
    q, s = torch.zeros(4, 24576, dtype=torch.uint8), torch.zeros(4, 384, dtype=BF)
    wt = torch.zeros(8, 2)
    with pytest.raises(ValueError, match="expert_q"):
        moe.moe_experts_w4(p, 128, x, idx, wt, q[:3], s, None, None, x, ws)
    with pytest.raises(ValueError, match="expert_scale"):
        moe.moe_experts_w4(p, 64, x, idx, wt, q, s, None, None, x, ws)
    with pytest.raises(ValueError, match="topk_w"):
        moe.moe_experts_w4(p, 128, x, idx, wt[:7], q, s, None, None, x, ws)


def test_packing_addresses_are_a_permutation():
    # every code and every scale of an expert belongs to exactly one weight
    import numpy as np
    I, H = 256, 384
    for group in (32, 64, 128):
        q = np.zeros(3 * I * H // 2, dtype=np.int64)
        for nib in (0, 1):
            (g, gs), (u, us), (d, ds) = ref.w4_unpack(q + (5 << (4 * nib)), np.arange(
                3 * I * H // group), I, H, group)
            got = sum(int((m == 5).sum()) for m in (g, u, d))
            assert got == q.size, (group, nib, got)
        seen = np.concatenate([gs.ravel(), us.ravel()])
        counts = np.bincount(seen, minlength=2 * I * H // group)
        assert (counts == group).all()
        assert (np.bincount(ds.ravel() - 2 * I * H // group) == group).all()
