"""4-bit experts on rows that are hard on block integers: outlier channels, zero rows
and blocks, tiny blocks, values on the borders of what is exact.

Bounds.  A row enters a product in blocks of 128 values as 16-bit integers times a
power of two a, amax/32384 <= a <= amax/16191, so a value is off by at most a/2.
Where the values below 1024 a of a block would lose more than 2^-9 of their 2-norm
to that, their remainders, at most a/2, enter as a second such integer: off by at
most 2^-14.9 of that again.  off_by() says which of the two holds, from that definition alone."""
import pytest
import torch

import operator_reference as ref
from sparse_moe_layer_06_b200 import moe
from test_gpu_w4 import draw_packed, draw_routing, problem, run_experts

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def split(v):
    """A block's integers t (not yet rounded: u) and scale a, in 64 bits."""
    b = v.reshape(v.shape[0], -1, 128)
    amax = b.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(amax)
    n = (e - 15 + (2 * m > 253 / 128).int()).clamp(min=-126)
    a = torch.ldexp(torch.ones_like(amax), n)
    u = b / a
    return u, a, n


def off_by(v, known):
    """Bound of each value's error.  known: v itself is what the kernel has (x); if not (h,
    which the kernel computes in fp32) the border may fall on the other side."""
    u, a, n = split(v)
    small = u.abs() < 1024
    rest = u - u.round()
    err, norm = (rest.square() * small).sum(-1), (u.square() * small).sum(-1)
    second = ((err > 2.0 ** -18 * norm * (1.001 if known else 2)) & (n[..., 0] > -126))[..., None]
    u2, a2, _ = split((rest * a).reshape(v.shape))
    if known:
        one, two = rest.abs() * a, (u2 - u2.round()).abs() * a2
    else:
        one = torch.where(u == 0, u, a / 2)
        two = one * 2.0 ** -14.9
    return torch.where(second, two, one).reshape(v.shape)


def bounded(x, mats, clip, group):
    """FFN of rows x in 64 bits and a bound on the kernel's error (the chain of fp32
    additions as in operator_reference.w4_ffn, twice its length: both integers).  The clamp
    only shrinks errors, |silu'| <= 1.1; exp, sum and quotient: 2^-20 of h."""
    gate, up, down = mats

    def product(v, dv, m):
        e = 2 * (m.shape[1] / group + 8 + 3) * 2.0 ** -24
        # (additions see the magnitudes of the limbs: 256 a beside |v|)
        big = v.abs().reshape(v.shape[0], -1, 128).amax(-1).repeat_interleave(128, -1) / 63
        return v @ m.T, dv @ m.abs().T + e * ((v.abs() + dv + big) @ m.abs().T)

    x = x.to(ref.F64)
    g, dg = product(x, off_by(x, True), gate)
    u, du = product(x, off_by(x, True), up)
    if clip > 0:
        g, u = g.clamp(-clip, clip), u.clamp(-clip, clip)
    silu = g * torch.sigmoid(g)
    h = silu * u
    dh = 1.1 * dg * (u.abs() + du) + silu.abs() * du + 2.0 ** -20 * h.abs()
    dh = dh + 2.0 ** -24 * (h.abs() + dh)
    # (the smallest fp32 and the smallest scale: 2^-126)
    return product(h, dh + off_by(h, False) * (1 + 2.0 ** -10) + 2.0 ** -126, down)


def layer(x, idx, w, experts, shared, clip, group):
    T, H = x.shape
    out, err, mag = (torch.zeros(T, H, dtype=ref.F64) for _ in range(3))
    for e, mats in enumerate(experts):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        if len(t):
            y, d = bounded(x[t], mats, clip, group)
            wt = w[t, j].to(ref.F64)[:, None]
            out.index_add_(0, t, wt * y)
            err.index_add_(0, t, wt.abs() * d)
            mag.index_add_(0, t, wt.abs() * y.abs())
    if shared is not None:
        y, d = bounded(x, shared, clip, group)
        out, err, mag = out + y, err + d, mag + y.abs()
    err = err + (idx.shape[1] + 3) * 2.0 ** -24 * (mag + err)
    return out, out.abs() * 2.0 ** -8 + err * (1 + 2.0 ** -8)


def zero_codes(p, q, columns, down=()):
    """The packed codes with weight 0 (code 8) at these columns of the gate and up
    matrices and of the down matrix, by the address of each weight."""
    q, gu = q.clone(), p.I * p.H
    for cols, K, base, tiles in ((columns, p.H, 0, p.I // 16), (down, p.I, gu, p.H // 32)):
        for k in cols:
            blk, kk = k // 128, k % 128
            b = kk // 32 * 8 + kk % 8 // 4 * 4 + kk % 2 * 2 + kk % 4 // 2
            part = q[:, base:base + tiles * (K // 128) * 2048].view(-1, tiles, K // 128, 2, 32, 32)
            for r in range(8):
                part[:, :, blk, :, r * 4 + kk % 32 // 8, b] = 0x88
    return q


# one to four rows a chunk, up to eight, up to sixteen; both dispatches
SIZES = [(1, 3, 2), (4, 3, 2), (24, 8, 2), (90, 6, 3), (260, 5, 2)]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("size", [30.0, 300.0, 3000.0, 1e6])
def test_small_values_beside_an_outlier(T, E, k, size, group):
    # a channel of each block is `size` times the others, in every second row, and no
    # weight looks at it: the rest of the row is all there is
    p = problem(T, 384, E, 256, k, 1, 10.0)
    outliers = [5, 128 + 77, 256 + 30]
    q, s = draw_packed(E, p, group, 50)
    sq, ss = draw_packed(1, p, group, 51)
    q, sq = zero_codes(p, q, outliers), zero_codes(p, sq, outliers)
    idx, w = draw_routing(T, E, k, 52)
    x = torch.randn(T, 384, generator=torch.Generator().manual_seed(53))
    x[::2, outliers] = size
    x = x.to(BF)
    out = run_experts(p, group, x, idx, w, q, s, sq, ss)
    want, bound = layer(x, idx, w, ref.w4_weights(q, s, 256, 384, group),
                        ref.w4_weights(sq, ss, 256, 384, group)[0], 10.0, group)
    ref.assert_within(out, want, bound, "out")
    # the rows' errors are those of the output's rounding: rms of a half step, 2^-8
    rel = (out.cpu().to(ref.F64) - want).square().sum(-1).sqrt() / want.square().sum(-1).sqrt()
    assert rel.max() < 2.0 ** -8


@pytest.mark.parametrize("T,group", [(3, 128), (3, 32), (7, 64), (13, 64), (13, 32), (13, 128)])
def test_marked_chunks_over_several_rounds(T, group):
    # 2560 pair tiles of gate and up: a CTA takes a chunk in two rounds, so the rows come
    # back after the second integers; then the down product with 320 blocks
    H, I = 128, 40960
    p = problem(T, H, 1, I, 1, 0, 0.0)
    q, s = draw_packed(1, p, group, 60, std=0.03)
    q = zero_codes(p, q, [40])
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(61))
    x[::2, 40] = 3000.0
    x = x.to(BF)
    idx, w = torch.zeros(T, 1, dtype=torch.int32), torch.rand(T, 1) + 0.1
    out = run_experts(p, group, x, idx, w, q, s, None, None)
    want, bound = layer(x, idx, w, ref.w4_weights(q, s, I, H, group), None, 0.0, group)
    ref.assert_within(out, want, bound, "out")


@pytest.mark.parametrize("T,E,k,group", [(300, 64, 8, 128), (70, 24, 3, 64), (5, 3, 2, 32),
                                         (120, 24, 3, 32)])
def test_chunks_with_and_without_marks_in_turn(T, E, k, group):
    # many small chunks to a CTA, those of every third expert with marked rows
    p = problem(T, 256, E, 128, k, 1, 10.0)
    q, s = draw_packed(E, p, group, 62)
    sq, ss = draw_packed(1, p, group, 63)
    q, sq = zero_codes(p, q, [3, 200]), zero_codes(p, sq, [3, 200])
    idx, w = draw_routing(T, E, k, 64)
    x = torch.randn(T, 256, generator=torch.Generator().manual_seed(65))
    clean = run_experts(p, group, x.to(BF), idx, w, q, s, sq, ss)
    hit = (idx % 3 == 0).any(-1) & (torch.arange(T) % 2 == 0)
    x[hit, 3], x[hit, 200] = 2000.0, -500.0
    x = x.to(BF)
    out = run_experts(p, group, x, idx, w, q, s, sq, ss)
    want, bound = layer(x, idx, w, ref.w4_weights(q, s, 128, 256, group),
                        ref.w4_weights(sq, ss, 128, 256, group)[0], 10.0, group)
    ref.assert_within(out, want, bound, "out")
    # the other rows are not touched by their neighbours' second integers
    assert hit.any() and not hit.all() and torch.equal(out[~hit], clean[~hit])
    assert torch.equal(out, run_experts(p, group, x, idx, w, q, s, sq, ss))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,E", [(3, 2), (11, 2), (40, 2)])
def test_small_values_of_h_beside_an_outlier(T, E, group):
    # one channel of h some thousand times the others, which the down weights do not see
    H, I = 256, 384
    p = problem(T, H, E, I, 1, 0, 0.0)
    g = torch.Generator().manual_seed(66)
    wt = torch.randn(E, 3, I, H, generator=g) * 0.05
    wt[:, :2, [7, 300]] *= 60.0
    q = torch.empty(E, 3 * I * H // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(E, 3 * I * H // group, dtype=BF, device="cuda")
    moe.moe_quantize_weights_w4(p, group, wt.to(BF).to("cuda"), q, s)
    q, s = zero_codes(p, q.cpu(), [], [7, 300]), s.cpu()
    idx, w = draw_routing(T, E, 1, 67)
    x = torch.randn(T, H, generator=g).to(BF)
    out = run_experts(p, group, x, idx, w, q, s, None, None)
    mats = ref.w4_weights(q, s, I, H, group)
    want, bound = layer(x, idx, w, mats, None, 0.0, group)
    ref.assert_within(out, want, bound, "out")
    rel = (out.cpu().to(ref.F64) - want).square().sum(-1).sqrt() / want.square().sum(-1).sqrt()
    assert rel.max() < 2.0 ** -8


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T", [8, 20])
def test_zero_tiny_and_large_rows(T, group):
    p = problem(T, 384, 2, 256, 2, 1, 10.0)
    q, s = draw_packed(2, p, group, 70)
    sq, ss = draw_packed(1, p, group, 71)
    idx, w = draw_routing(T, 2, 2, 72)
    x = torch.randn(T, 384, generator=torch.Generator().manual_seed(73))
    x[0] = 0.0                          # no value
    x[1, 128:256] = 0.0                 # a block without
    x[2] *= 2.0 ** -100                 # below the smallest block that keeps 15 bits
    x[3, :128] *= 2.0 ** -60            # a block far below its neighbours
    x[4] = 0.0
    x[4, 200] = 1.5                     # one value
    x[5] *= 1e30
    x[6] = -0.0
    x[7] = torch.finfo(torch.float32).tiny
    x = x.to(BF)
    out = run_experts(p, group, x, idx, w, q, s, sq, ss)
    want, bound = layer(x, idx, w, ref.w4_weights(q, s, 256, 384, group),
                        ref.w4_weights(sq, ss, 256, 384, group)[0], 10.0, group)
    ref.assert_within(out, want, bound, "out")
    assert not out[0].any() and not out[6].any()


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("top", [252, 253, 254, 255])
def test_what_is_exact(group, top):
    # the largest mantissas of a block on both sides of the doubled scale; beside them values
    # down to 2^-6 of it, which are exact, and to 2^-8, which need not be
    p = problem(4, 128, 1, 128, 1, 0, 0.0)
    q, s = draw_packed(1, p, group, 74)
    m = torch.arange(128, 256).float()
    x = torch.zeros(4, 128)
    x[0] = m * 2.0 ** -6                # top / 64 and above (but for the smallest mantissas)
    x[0, : top - 128] = m[: top - 128] * 2.0 ** -5
    x[1] = m * 2.0 ** -7
    x[2] = m * 2.0 ** -8
    x[3] = -m * 2.0 ** -3
    x[:, 60] = float(top)
    assert torch.equal(x.to(BF).float(), x) and (x[0].abs() >= top / 64).all()
    assert not off_by(x[:1].to(ref.F64), True).any() and not off_by(x[3:].to(ref.F64), True).any()
    idx, w = torch.zeros(4, 1, dtype=torch.int32), torch.ones(4, 1)
    out = run_experts(p, group, x.to(BF), idx, w, q, s, None, None)
    want, bound = layer(x.to(BF), idx, w, ref.w4_weights(q, s, 128, 128, group), None, 0.0, group)
    ref.assert_within(out, want, bound, "out")


@pytest.mark.parametrize("T", [4, 40, 300])
def test_replays_on_rows_with_and_without_outliers(T):
    # the marks are the rows' as they are at the replay, in one workspace, and two calls at
    # once do not meet
    p = problem(T, 384, 6, 256, 2, 1, 10.0)
    q, s = draw_packed(6, p, 64, 75)
    sq, ss = draw_packed(1, p, 64, 76)
    idx, w = draw_routing(T, 6, 2, 77)
    plain = torch.randn(T, 384, generator=torch.Generator().manual_seed(78))
    hard = plain.clone()
    hard[::2, 7], hard[::3, 300] = 2000.0, -700.0
    batches = [plain.to(BF), hard.to(BF), plain.to(BF), hard.to(BF)]
    want = [run_experts(p, 64, x, idx, w, q, s, sq, ss) for x in batches]
    d = [t.to("cuda") for t in (idx, w, q, s, sq, ss)]
    x, out = torch.empty_like(batches[0], device="cuda"), torch.empty_like(want[0])
    ws = moe.alloc_workspace(p, moe.MOE_CALL_EXPERTS_W4)
    x.copy_(batches[0])
    call = lambda: moe.moe_experts_w4(p, 64, x, *d, out, ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for b, y in zip(batches, want):
        x.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, y)
    del graph
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = [(b.to("cuda"), torch.empty_like(out), moe.alloc_workspace(p, moe.MOE_CALL_EXPERTS_W4))
            for b in batches[:2]]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, (xs, o, wsp) in zip(streams, sets):
            moe.moe_experts_w4(p, 64, xs, *d, o, wsp, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(o, y) for (_, o, _), y in zip(sets, want))
