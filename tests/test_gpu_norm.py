"""Residual addition + RMS norm (with E4M3 codes) and its backward pass against
the 64-bit forms in operator_reference (which states the bounds)."""
import pytest
import torch

import operator_reference as ref
from sparse_moe_layer_06_b200 import moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def problem(T, H, dtype):
    return moe.MoEProblem(T=T, H=H, E=4, I=64, top_k=1, num_shared=0, routed_scale=1.0,
                          clip_limit=0.0, dtype=dtype)


def draw(T, H, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, H, generator=g) * std).to(dtype)


def run_norm(x, res, w, eps, codes=False, want_y=True):
    T, H = x.shape
    p = problem(T, H, x.dtype)
    d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    ro = None if res is None else torch.full((T, H), float("nan"), dtype=x.dtype, device=DEV)
    y = torch.full((T, H), float("nan"), dtype=x.dtype, device=DEV) if want_y else None
    q = torch.full((T, H), 255, dtype=torch.uint8, device=DEV) if codes else None
    s = torch.full((T,), float("nan"), device=DEV) if codes else None
    moe.moe_add_rmsnorm(p, d(x), d(res), d(w), eps, ro, y, q, s)
    torch.cuda.synchronize()
    return ro, y, q, s


# warp-per-row widths, one and several vectors per thread, odd multiples of 64,
# widths that leave threads without a vector, the widest row
SHAPES = [(1, 64), (5, 64), (7, 192), (3, 1024), (1, 1088), (33, 1984), (2, 6144), (1, 7168),
          (4, 7616), (2, 16384), (1000, 320)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_matches_64_bits(T, H, dtype, residual):
    x = draw(T, H, dtype, 1)
    res = draw(T, H, dtype, 2, 3.0) if residual else None
    w = draw(1, H, dtype, 3, 0.2)[0] + 1
    ro, y, _, _ = run_norm(x, res, w, 1e-6)
    s, yr, _ = ref.norm(x, res, w, 1e-6)
    ref.assert_within(y, yr, ref.norm_y_bound(yr, dtype), "y")
    if residual:
        # the fp32 sum, then the row type
        ref.assert_within(ro, s, s.abs() * (ref.HALF_STEP[dtype] + 2.0 ** -24 * 1.01), "residual")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,H", [(1, 64), (37, 320), (3, 6144), (1, 16384)])
@pytest.mark.parametrize("want_y", [True, False])
def test_codes_are_those_of_the_rounded_rows(dtype, T, H, want_y):
    x, res = draw(T, H, dtype, 4), draw(T, H, dtype, 5, 3.0)
    x[0] = 0
    res[0] = 0  # a row of zeros: scale 1, codes 0
    w = draw(1, H, dtype, 6, 0.5)[0]
    _, y, _, _ = run_norm(x, res, w, 1e-5)
    _, y2, q, s = run_norm(x, res, w, 1e-5, codes=True, want_y=want_y)
    if want_y:
        assert torch.equal(y, y2)
    amax = y.float().abs().amax(-1)
    # s = 2^n with the smallest n for which 448 * 2^n >= amax
    live = amax > 0
    assert torch.equal(s[~live], torch.ones_like(s[~live]))
    assert (s[live] * 448 >= amax[live]).all() and (s[live] / 2 * 448 < amax[live]).all()
    assert (torch.frexp(s)[0] == 0.5).all()
    want = (y.float() / s[:, None]).to(torch.float8_e4m3fn)
    assert torch.equal(q, want.view(torch.uint8))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_eps_dominates_tiny_rows_and_zero_eps(dtype):
    x = draw(4, 256, dtype, 7, 1e-4)
    w = draw(1, 256, dtype, 8)[0]
    for eps in (1e-2, 0.0):
        _, y, _, _ = run_norm(x, None, w, eps)
        _, yr, _ = ref.norm(x, None, w, eps)
        ref.assert_within(y, yr, ref.norm_y_bound(yr, dtype), f"eps {eps}")


# several rows per CTA pass through the ring of a wide row's copies, the last CTAs
# with one row fewer; one, two and three vectors per thread
@pytest.mark.parametrize("dtype,T,H", [(BF, 2503, 1152), (BF, 2503, 2112), (BF, 2503, 9024),
                                       (BF, 445, 16384), (F32, 2503, 1152), (F32, 2503, 3136),
                                       (F32, 445, 16384)])
def test_many_wide_rows(dtype, T, H):
    x, res = draw(T, H, dtype, 50), draw(T, H, dtype, 51, 3.0)
    w = draw(1, H, dtype, 52, 0.2)[0] + 1
    ro, y, q, s = run_norm(x, res, w, 1e-6, codes=True)
    sr, yr, _ = ref.norm(x, res, w, 1e-6)
    ref.assert_within(y, yr, ref.norm_y_bound(yr, dtype), "y")
    ref.assert_within(ro, sr, sr.abs() * (ref.HALF_STEP[dtype] + 2.0 ** -24 * 1.01), "residual")
    want = (y.float() / s[:, None]).to(torch.float8_e4m3fn)
    assert torch.equal(q, want.view(torch.uint8))
    dy, dres = draw(T, H, dtype, 53, 0.01), draw(T, H, dtype, 54, 0.01)
    dx, dw = run_backward(dy, dres, x, w, 1e-6)
    dxr, dwr, mx, mw = ref.norm_backward(dy, dres, x, w, 1e-6)
    ref.assert_within(dx, dxr, ref.norm_dx_bound(dxr, mx, dtype), "dx")
    ref.assert_within(dw, dwr, ref.norm_dw_bound(mw, T), "dweight")
    # the same rows in place, and alone
    xd, rd = x.to(DEV), res.to(DEV)
    moe.moe_add_rmsnorm(problem(T, H, dtype), xd, rd, w.to(DEV), 1e-6, rd, xd)
    assert torch.equal(xd, y) and torch.equal(rd, ro)
    alone = run_norm(x[T - 1:], res[T - 1:], w, 1e-6)[1]
    assert torch.equal(alone[0], y[T - 1])


def test_infinities_and_nans_stay_in_their_rows():
    x = draw(4, 512, BF, 9)
    clean = run_norm(x, None, torch.ones(512, dtype=BF), 1e-6, codes=True)
    x[1, 3] = float("inf")
    x[2, 500] = float("nan")
    _, y, q, s = run_norm(x, None, torch.ones(512, dtype=BF), 1e-6, codes=True)
    for t in (0, 3):
        assert torch.equal(y[t], clean[1][t]) and torch.equal(q[t], clean[2][t])
    assert torch.isnan(y[1, 3]) and (y[1, :3] == 0).all()
    assert torch.isnan(y[2]).all()
    assert (q[2] == 0x7f).all() and (s > 0).all()


def test_in_place_rows():
    T, H = 19, 640
    x, res, w = draw(T, H, BF, 10), draw(T, H, BF, 11, 3.0), draw(1, H, BF, 12)[0]
    ro, y, _, _ = run_norm(x, res, w, 1e-6)
    xd, rd = x.to(DEV), res.to(DEV)
    moe.moe_add_rmsnorm(problem(T, H, BF), xd, rd, w.to(DEV), 1e-6, rd, xd)
    assert torch.equal(xd, y) and torch.equal(rd, ro)


def test_rows_behind_the_batch_are_left():
    x = draw(9, 128, BF, 13).to(DEV)
    y = torch.full((9, 128), 7.0, dtype=BF, device=DEV)
    moe.moe_add_rmsnorm(problem(5, 128, BF), x, None, torch.ones(128, dtype=BF, device=DEV), 1e-6,
                        None, y)
    assert (y[5:] == 7.0).all() and not (y[:5] == 7.0).all()


def run_backward(dy, dres, h, w, eps, ws=None, stream=None):
    T, H = dy.shape
    p = problem(T, H, dy.dtype)
    d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    dx = torch.full((T, H), float("nan"), dtype=dy.dtype, device=DEV)
    dw = torch.full((H,), float("nan"), device=DEV)
    if ws is None:
        ws = moe.alloc_workspace(p, moe.MOE_CALL_ADD_RMSNORM_BACKWARD)
        ws.fill_(0xff)  # nothing of it is read before it is written
    moe.moe_add_rmsnorm_backward(p, d(dy), d(dres), d(h), d(w), eps, dx, dw, ws, stream)
    torch.cuda.synchronize()
    return dx, dw


@pytest.mark.parametrize("T,H", SHAPES + [(445, 128), (889, 64)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("residual", [False, True])
def test_backward_matches_64_bits(T, H, dtype, residual):
    dy, h = draw(T, H, dtype, 14, 0.01), draw(T, H, dtype, 15, 3.0)
    dres = draw(T, H, dtype, 16, 0.01) if residual else None
    w = draw(1, H, dtype, 17, 0.2)[0] + 1
    dx, dw = run_backward(dy, dres, h, w, 1e-6)
    dxr, dwr, mx, mw = ref.norm_backward(dy, dres, h, w, 1e-6)
    ref.assert_within(dx, dxr, ref.norm_dx_bound(dxr, mx, dtype), "dx")
    ref.assert_within(dw, dwr, ref.norm_dw_bound(mw, T), "dweight")


def test_backward_against_differences():
    # central differences of sum(dy * y) + sum(dres * residual_out) in fp64: the
    # quotient is off by d^2/6 of the third derivative (about 1e-9 here at
    # d = 1e-4), far below the kernel's own bound
    T, H, d = 5, 128, 1e-4
    x, dy, dres = (draw(T, H, F32, 20 + i) for i in range(3))
    w = draw(1, H, F32, 23, 0.2)[0] + 1
    dx, dw = run_backward(dy, dres, x, w, 1e-5)

    def value(xx, ww):
        s, y, _ = ref.norm(xx, None, ww, 1e-5)
        return (dy.to(ref.F64) * y + dres.to(ref.F64) * s).sum()

    g = torch.Generator().manual_seed(24)
    for _ in range(4):
        v = torch.randn(T, H, generator=g, dtype=ref.F64)
        u = torch.randn(H, generator=g, dtype=ref.F64)
        x64, w64 = x.to(ref.F64), w.to(ref.F64)
        num_x = (value(x64 + d * v, w64) - value(x64 - d * v, w64)) / (2 * d)
        num_w = (value(x64, w64 + d * u) - value(x64, w64 - d * u)) / (2 * d)
        _, _, mx, mw = ref.norm_backward(dy, dres, x, w, 1e-5)
        bx = ((ref.norm_dx_bound(dx.cpu().to(ref.F64), mx, F32)) * v.abs()).sum() + 1e-6
        bw = (ref.norm_dw_bound(mw, T) * u.abs()).sum() + 1e-6
        assert abs((dx.cpu().to(ref.F64) * v).sum() - num_x) <= bx
        assert abs((dw.cpu().to(ref.F64) * u).sum() - num_w) <= bw


def test_backward_in_place_reproducible_and_empty():
    T, H = 700, 1024
    dy, h, dres = draw(T, H, BF, 30), draw(T, H, BF, 31), draw(T, H, BF, 32)
    w = draw(1, H, BF, 33)[0]
    dx, dw = run_backward(dy, dres, h, w, 1e-6)
    dx2, dw2 = run_backward(dy, dres, h, w, 1e-6)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    p = problem(T, H, BF)
    for inplace in ("dy", "dres"):
        a = {"dy": dy.to(DEV), "dres": dres.to(DEV)}
        dw3 = torch.empty(H, device=DEV)
        moe.moe_add_rmsnorm_backward(p, a["dy"], a["dres"], h.to(DEV), w.to(DEV), 1e-6, a[inplace],
                                     dw3, moe.alloc_workspace(p, moe.MOE_CALL_ADD_RMSNORM_BACKWARD))
        assert torch.equal(a[inplace], dx) and torch.equal(dw3, dw)
    e = torch.empty(0, H, dtype=BF, device=DEV)
    dw4 = torch.full((H,), 3.0, device=DEV)
    p0 = problem(0, H, BF)
    moe.moe_add_rmsnorm_backward(p0, e, None, e, w.to(DEV), 1e-6, e, dw4,
                                 moe.alloc_workspace(p0, moe.MOE_CALL_ADD_RMSNORM_BACKWARD))
    moe.moe_add_rmsnorm(p0, e, None, w.to(DEV), 1e-6, None, e)
    assert (dw4 == 0).all()


def test_on_a_side_stream():
    T, H = 300, 2048
    x, w = draw(T, H, BF, 40).to(DEV), draw(1, H, BF, 41)[0].to(DEV)
    want = run_norm(x.cpu(), None, w.cpu(), 1e-6)[1]
    side = torch.cuda.Stream()
    y = torch.empty_like(x)
    side.wait_stream(torch.cuda.current_stream())
    moe.moe_add_rmsnorm(problem(T, H, BF), x, None, w, 1e-6, None, y, stream=side)
    side.synchronize()
    assert torch.equal(y, want)


def test_rows_past_the_32_bit_offset():
    # 2^31 elements and more: the last rows are those of a small batch
    T, H = 131075, 16384
    g = torch.Generator(device=DEV).manual_seed(60)
    tail = torch.randn(5, H, generator=g, device=DEV).to(BF)
    w = torch.rand(H, generator=g, device=DEV).to(BF)
    x = torch.zeros(T, H, dtype=BF, device=DEV)
    x[T - 5:] = tail
    y = torch.empty_like(x)
    moe.moe_add_rmsnorm(problem(T, H, BF), x, x, w, 1e-6, None, y)
    small = run_norm(tail, tail, w, 1e-6)[1]
    assert torch.equal(y[T - 5:], small) and not y[:T - 5].any()
    p = problem(T, H, BF)
    dw = torch.empty(H, device=DEV)
    moe.moe_add_rmsnorm_backward(p, x, None, x, w, 1e-6, y, dw,
                                 moe.alloc_workspace(p, moe.MOE_CALL_ADD_RMSNORM_BACKWARD))
    dx, _ = run_backward(tail, None, tail, w, 1e-6)
    assert torch.equal(y[T - 5:], dx) and not y[:T - 5].any()
    _, dwr, _, mw = ref.norm_backward(tail.cpu(), None, tail.cpu(), w.cpu(), 1e-6)
    ref.assert_within(dw, dwr, ref.norm_dw_bound(mw, T), "dweight")
