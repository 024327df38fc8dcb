"""Widths of the norm from the smallest to the largest, and every kernel instance of
it with its ring used several times over, against the 64-bit forms of operator_reference (on the GPU)."""
import os
import re

import pytest
import torch

import operator_reference as ref
from sparse_moe_layer_06_b200 import moe

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
SOURCE = os.path.join(os.path.dirname(__file__), "..", "sparse_moe_layer_06_b200", "csrc",
                      "ops_api.cu")


def constants():
    with open(SOURCE) as f:
        src = f.read()
    get = lambda n: int(re.search(rf"\b{n} = (\d+)", src).group(1))  # noqa: E731
    return {n: get(n) for n in ("kNormThreadsPerSM", "kNormBackThreadsPerSM", "kNormTwo",
                                "kNormBackTwo")} | {"ring": 1024 * int(
                                    re.search(r"kRingBytesPerSM = (\d+) \* 1024", src).group(1))}


def instance(c, H, dtype, inputs, backward):
    """(vectors per thread, ring depth, most threads), and CTAs per SM, as the launch
    chooses them; None for the short rows, which have no ring."""
    size = 2 if dtype == BF else 4
    nv = H * size // 16
    two = c["kNormBackTwo" if backward else "kNormTwo"]
    vpt = 2 if nv <= two else 4
    threads = max(32, (-(-nv // vpt) + 31) // 32 * 32)
    ctas = max(1, min(8, c["kNormBackThreadsPerSM" if backward else "kNormThreadsPerSM"] // threads))
    rows = c["ring"] // ctas // (inputs * H * size)
    depth = 4 if rows >= 4 else 2 if rows >= 2 else 1
    if backward:
        return (vpt, depth, 512 if threads <= 512 else 1024), ctas
    if nv <= 128:
        return None, ctas
    return (vpt, depth, 1024 if vpt == 4 and dtype == F32 else 512), ctas


def cases(dtype, backward):
    """First and last width of each instance and number of inputs: what a launch can take."""
    c, found = constants(), {}
    for H in range(64, 16385, 64):
        for inputs in ((2, 3) if backward else (1, 2)):
            key, ctas = instance(c, H, dtype, inputs, backward)
            if key:
                found.setdefault(key, {}).setdefault(inputs, []).append((H, ctas))
    return found


def test_no_width_needs_an_instance_that_is_not_there():
    # the instances of the launch code; a threshold that moves has to move them too
    want = {(BF, False): {(2, 4, 512), (4, 4, 512), (4, 2, 512)},
            (F32, False): {(2, 4, 512), (4, 4, 1024), (4, 2, 1024), (4, 1, 1024)},
            (BF, True): {(2, 4, 512), (2, 4, 1024), (2, 2, 1024)},
            (F32, True): {(2, 4, 512), (2, 4, 1024), (2, 2, 1024), (4, 2, 1024), (4, 1, 1024)}}
    for (dtype, backward), keys in want.items():
        assert set(cases(dtype, backward)) == keys, (dtype, backward)


def rows(T, H, dtype, seed, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(T, H, generator=g, device=DEV) * std).to(dtype)


def within(got, want, bound, what):
    assert torch.isfinite(got).all(), what
    assert ((got.to(ref.F64) - want).abs() <= bound).all(), what


def problem(T, H, dtype):
    return moe.MoEProblem(T=T, H=H, E=1, I=64, top_k=1, num_shared=0, routed_scale=1.0,
                          clip_limit=0.0, dtype=dtype)


def forward(T, H, dtype, residual):
    x, w = rows(T, H, dtype, 1), rows(1, H, dtype, 2, 0.2)[0] + 1
    res = rows(T, H, dtype, 3, 3.0) if residual else None
    y = torch.full((T, H), float("nan"), dtype=dtype, device=DEV)
    ro = torch.full_like(y, float("nan")) if residual else None
    moe.moe_add_rmsnorm(problem(T, H, dtype), x, res, w, 1e-6, ro, y)
    s, want, _ = ref.norm(x, res, w, 1e-6)
    within(y, want, ref.norm_y_bound(want, dtype), (H, "y"))
    if residual:
        within(ro, s, s.abs() * (ref.HALF_STEP[dtype] + 2.0 ** -24 * 1.01), (H, "residual"))


def backward(T, H, dtype, residual):
    dy, h = rows(T, H, dtype, 4, 0.01), rows(T, H, dtype, 5, 3.0)
    dres = rows(T, H, dtype, 6, 0.01) if residual else None
    w = rows(1, H, dtype, 7, 0.2)[0] + 1
    p = problem(T, H, dtype)
    dx, dw = torch.full_like(dy, float("nan")), torch.full((H,), float("nan"), device=DEV)
    ws = moe.alloc_workspace(p, moe.MOE_CALL_ADD_RMSNORM_BACKWARD)
    ws.fill_(0xff)
    moe.moe_add_rmsnorm_backward(p, dy, dres, h, w, 1e-6, dx, dw, ws)
    want, dwr, mx, mw = ref.norm_backward(dy, dres, h, w, 1e-6)
    within(dx, want, ref.norm_dx_bound(want, mx, dtype), (H, "dx"))
    within(dw, dwr, ref.norm_dw_bound(mw, T), (H, "dweight"))


@pytest.mark.gpu
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_widths_from_the_smallest_to_the_largest(dtype, residual):
    for H in (*range(64, 16384, 128), 16384):  # odd multiples of 64
        forward(3, H, dtype, residual)
        backward(3, H, dtype, residual)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("back", [False, True])
def test_every_instance_with_many_rows_to_a_cta(dtype, back):
    for key, by_inputs in cases(dtype, back).items():
        for inputs, widths in by_inputs.items():
            for H, ctas in {widths[0], widths[-1]}:
                # six rows to each CTA, the last ones five: every slot of the ring is
                # filled again, and dweight adds up over rows
                (backward if back else forward)(148 * ctas * 6 - 5, H, dtype,
                                                inputs == (3 if back else 2))
