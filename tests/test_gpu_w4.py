"""4-bit expert weights: the encoder bit for bit, the experts' products and the
whole layer against the 64-bit forms in operator_reference (which states the
bounds)."""
import numpy as np
import pytest
import torch

import operator_reference as ref
import oracle
from parity_util import check_routing, to_cpu_inputs
from sparse_moe_layer_06_b200 import moe
from sparse_moe_layer_06_b200.workloads import MoEConfig, make_inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def problem(T, H, E, I, k, shared=0, clip=10.0, dtype=BF):
    return moe.MoEProblem(T=T, H=H, E=E, I=I, top_k=k, num_shared=shared, routed_scale=2.827,
                          clip_limit=clip, dtype=dtype)


def encode(p, w, group):
    n, per = w.shape[0], 3 * p.I * p.H
    q = torch.empty(n, per // 2, dtype=torch.uint8, device=DEV)
    s = torch.empty(n, per // group, dtype=BF, device=DEV)
    moe.moe_quantize_weights_w4(p, group, w.to(DEV), q, s)
    torch.cuda.synchronize()
    return q, s


def draw_packed(n, p, group, seed, std=0.05):
    """Random packed weights: any bytes are codes."""
    g = torch.Generator().manual_seed(seed)
    per = 3 * p.I * p.H
    q = torch.randint(0, 256, (n, per // 2), generator=g, dtype=torch.int32).to(torch.uint8)
    s = (std / 4 * (0.5 + torch.rand(n, per // group, generator=g))).to(BF)
    return q, s


def draw_routing(T, E, k, seed):
    g = torch.Generator().manual_seed(seed)
    idx = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    return idx, torch.rand(T, k, generator=g) + 0.1


def run_experts(p, group, x, idx, w, q, s, sq, ss, status=0, poison=True):
    d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    ws = moe.alloc_workspace(p, moe.MOE_CALL_EXPERTS_W4)
    if poison:
        ws[256:] = 0xff  # nothing of it is read before it is written
    out = torch.full((p.T, p.H), float("nan"), dtype=BF, device=DEV)
    moe.moe_experts_w4(p, group, d(x), d(idx), d(w), d(q), d(s), d(sq), d(ss), out, ws)
    torch.cuda.synchronize()
    assert moe.moe_read_device_status(ws) == status
    return out


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("H,I", [(128, 128), (384, 256)])
def test_encoder_bit_exact(dtype, group, H, I):
    g = torch.Generator().manual_seed(1)
    w = torch.randn(3, 3, I, H, generator=g) * 0.02
    w[0, 0, 3] = 0.0                                   # groups of zeros
    w[0, 1, 5, 17] = 3e4                               # one value swamps its group
    w[1, 0, 7] *= 1e-30                                # small scales
    w[1, 2, :, 9] *= 1e-41                             # scales that bf16 rounds to nothing
    w[2, 1, 11, :15] = torch.arange(-7, 8) * 0.5       # multiples of the scale, and
    w[2, 1, 11, 15:32] = torch.arange(17) * 0.25 - 2   # halves of it (ties)
    w[2, 1, 11, 16] = 7 * 0.5
    w = w.to(dtype)
    p = problem(1, H, 3, I, 1, dtype=dtype)
    q, s = encode(p, w, group)
    for e in range(3):
        mats = ref.w4_unpack(q[e].cpu().numpy().astype(np.int64), s[e].float().cpu().numpy(), I,
                             H, group)
        for m, src in zip(mats, (w[e, 0], w[e, 1], w[e, 2].T)):
            code, scale = ref.w4_encode(src.contiguous(), group)
            assert np.array_equal(m[0], code)
            assert np.array_equal(m[1], np.repeat(scale, group, axis=-1))


def test_encoder_marks_groups_that_are_not_finite():
    w = torch.randn(1, 3, 128, 128)
    w[0, 0, 4, 40], w[0, 2, 100, 7] = float("nan"), float("inf")
    p = problem(1, 128, 1, 128, 1)
    q, s = encode(p, w.to(BF), 32)
    gate, up, down = ref.w4_weights(q, s, 128, 128, 32)[0]
    assert torch.isnan(gate[4, 32:64]).all() and torch.isfinite(gate[4, :32]).all()
    assert torch.isnan(down[7, 96:]).all() and int(torch.isnan(down).sum()) == 32
    assert torch.isfinite(up).all() and int(torch.isnan(gate).sum()) == 32


def test_encoding_error_is_half_a_step():
    w = (torch.randn(2, 3, 128, 256) * 0.02).to(BF)
    p = problem(1, 256, 2, 128, 1)
    q, s = encode(p, w, 64)
    for e, (gate, up, down) in enumerate(ref.w4_weights(q, s, 128, 256, 64)):
        for m, src in ((gate, w[e, 0]), (up, w[e, 1]), (down, w[e, 2].T)):
            src = src.to(ref.F64)
            big = src.reshape(*src.shape[:-1], -1, 64).abs().amax(-1).repeat_interleave(64, -1)
            # half a step, and what the scale's rounding takes off the largest value
            assert ((m - src).abs() <= big / 7 * (1 + 2.0 ** -8) * 0.5 + big * 2.0 ** -8).all()


# one token; rows per expert that take each column-tile width, with one chunk
# and several; experts without rows; every expert; one expert for all; K of one
# block and of odd and even numbers of blocks; all group sizes
CASES = [
    (1, 128, 1, 128, 1, 0, 128), (1, 256, 8, 128, 2, 1, 64), (2, 384, 16, 256, 4, 1, 32),
    (9, 256, 4, 384, 2, 0, 128), (17, 128, 5, 128, 5, 1, 32), (33, 256, 2, 256, 1, 1, 64),
    (70, 384, 3, 128, 3, 0, 128), (40, 640, 8, 384, 2, 1, 32), (260, 128, 4, 128, 2, 1, 64),
    (300, 128, 64, 128, 8, 0, 128), (64, 256, 16, 128, 6, 1, 32),
]


@pytest.mark.parametrize("T,H,E,I,k,shared,group", CASES)
@pytest.mark.parametrize("clip", [10.0, 0.0])
def test_experts_match_64_bits(T, H, E, I, k, shared, group, clip):
    p = problem(T, H, E, I, k, shared, clip)
    q, s = draw_packed(E, p, group, 2)
    sq, ss = draw_packed(1, p, group, 3) if shared else (None, None)
    idx, w = draw_routing(T, E, k, 4)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(5)).to(BF)
    out = run_experts(p, group, x, idx, w, q, s, sq, ss)
    sh = ref.w4_weights(sq, ss, I, H, group)[0] if shared else None
    want, bound = ref.w4_layer(x, idx, w, ref.w4_weights(q, s, I, H, group), sh, clip, group)
    ref.assert_within(out, want, bound, "out")


# contractions so long that a chunk holds fewer rows than a column tile, down to
# one, with the rows behind it read but not stored
@pytest.mark.parametrize("T,H,I,group", [(21, 20480, 128, 64), (19, 128, 20480, 32),
                                         (5, 65536, 128, 128), (40, 128, 65536, 128)])
def test_long_contractions(T, H, I, group):
    p = problem(T, H, 2, I, 1, 1, 0.0)
    q, s = draw_packed(2, p, group, 30, std=0.01)
    sq, ss = draw_packed(1, p, group, 31, std=0.01)
    idx, w = draw_routing(T, 2, 1, 32)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(33)).to(BF)
    out = run_experts(p, group, x, idx, w, q, s, sq, ss)
    sh = ref.w4_weights(sq, ss, I, H, group)[0]
    want, bound = ref.w4_layer(x, idx, w, ref.w4_weights(q, s, I, H, group), sh, 0.0, group)
    ref.assert_within(out, want, bound, "out")


def test_codes_past_4_gigabytes():
    # the last expert's codes start behind byte 2^32: the same expert alone gives
    # the same rows (E = 16 of 302 MB each; the products' order does not depend on E)
    H, I, E = 16384, 12288, 16
    per = 3 * I * H
    g = torch.Generator(device=DEV).manual_seed(40)
    q = torch.randint(0, 256, (E, per // 2), generator=g, dtype=torch.uint8, device=DEV)
    s = ((0.5 + torch.rand(E, per // 128, generator=g, device=DEV)) * 0.002).to(BF)
    assert (E - 1) * (per // 2) > 1 << 32
    x = torch.randn(3, H, generator=g, device=DEV).to(BF)
    w = torch.rand(3, 1, generator=g, device=DEV)
    outs = []
    for n, e in ((E, E - 1), (1, 0)):
        idx = torch.full((3, 1), e, dtype=torch.int32, device=DEV)
        p = problem(3, H, n, I, 1)
        outs.append(run_experts(p, 128, x, idx, w, q[E - n:], s[E - n:], None, None))
    assert torch.equal(*outs) and torch.isfinite(outs[0]).all() and (outs[0] != 0).any()


def test_clamp_saturates():
    p = problem(12, 256, 4, 128, 2, 1, 2.5)
    q, s = draw_packed(4, p, 128, 6, std=2.0)
    sq, ss = draw_packed(1, p, 128, 7, std=2.0)
    idx, w = draw_routing(12, 4, 2, 8)
    x = torch.randn(12, 256, generator=torch.Generator().manual_seed(9)).to(BF)
    out = run_experts(p, 128, x, idx, w, q, s, sq, ss)
    want, bound = ref.w4_layer(x, idx, w, ref.w4_weights(q, s, 128, 256, 128),
                               ref.w4_weights(sq, ss, 128, 256, 128)[0], 2.5, 128)
    ref.assert_within(out, want, bound, "out")


@pytest.mark.parametrize("T", [5, 300])
def test_bad_experts_add_nothing(T):
    # both forms of the dispatch: an expert out of range sets the error word and
    # its assignment counts as absent
    p = problem(T, 128, 6, 128, 2)
    q, s = draw_packed(6, p, 64, 10)
    idx, w = draw_routing(T, 6, 2, 11)
    x = torch.randn(T, 128, generator=torch.Generator().manual_seed(12)).to(BF)
    bad = idx.clone()
    bad[1, 0], bad[T - 1, 1] = -1, 6
    out = run_experts(p, 64, x, bad, w, q, s, None, None, status=moe.MOE_ERR_BAD_INDEX)
    want, bound = ref.w4_layer(x, bad, w, ref.w4_weights(q, s, 128, 128, 64), None, 10.0, 64)
    ref.assert_within(out, want, bound, "out")


def test_an_expert_listed_twice_is_reported():
    p = problem(3, 128, 4, 128, 2)
    q, s = draw_packed(4, p, 128, 13)
    idx = torch.tensor([[0, 1], [2, 2], [3, 0]], dtype=torch.int32)
    w = torch.ones(3, 2)
    x = torch.randn(3, 128, generator=torch.Generator().manual_seed(14)).to(BF)
    out = run_experts(p, 128, x, idx, w, q, s, None, None, status=moe.MOE_ERR_BAD_INDEX)
    want, bound = ref.w4_layer(x, idx, w, ref.w4_weights(q, s, 128, 128, 128), None, 10.0, 128)
    keep = [0, 2]
    ref.assert_within(out[keep], want[keep], bound[keep], "the other rows")


def test_infinite_and_nan_rows_stay_theirs():
    T = 20
    p = problem(T, 256, 4, 128, 2, 1)
    q, s = draw_packed(4, p, 32, 15)
    sq, ss = draw_packed(1, p, 32, 16)
    idx, w = draw_routing(T, 4, 2, 17)
    x = torch.randn(T, 256, generator=torch.Generator().manual_seed(18)).to(BF)
    clean = run_experts(p, 32, x, idx, w, q, s, sq, ss)
    x[3, 5], x[11, 200] = float("nan"), float("inf")
    out = run_experts(p, 32, x, idx, w, q, s, sq, ss)
    keep = [t for t in range(T) if t not in (3, 11)]
    assert torch.equal(out[keep], clean[keep])
    assert torch.isnan(out[3]).all()


@pytest.mark.parametrize("group", [32, 64, 128])
def test_infinite_and_nan_rows_in_chunks_of_up_to_four(group):
    p = problem(4, 256, 3, 128, 2, 1)
    q, s = draw_packed(3, p, group, 34)
    sq, ss = draw_packed(1, p, group, 35)
    idx, w = draw_routing(4, 3, 2, 36)
    x = torch.randn(4, 256, generator=torch.Generator().manual_seed(37)).to(BF)
    clean = run_experts(p, group, x, idx, w, q, s, sq, ss)
    x[1, 5], x[2, 200] = float("nan"), float("-inf")
    out = run_experts(p, group, x, idx, w, q, s, sq, ss)
    assert torch.equal(out[[0, 3]], clean[[0, 3]])
    assert torch.isnan(out[[1, 2]]).all()


def test_reproducible_and_rows_behind_the_batch_left():
    p = problem(50, 384, 8, 256, 3, 1)
    q, s = draw_packed(8, p, 64, 19)
    sq, ss = draw_packed(1, p, 64, 20)
    idx, w = draw_routing(50, 8, 3, 21)
    x = torch.randn(50, 384, generator=torch.Generator().manual_seed(22)).to(BF)
    a = run_experts(p, 64, x, idx, w, q, s, sq, ss)
    b = run_experts(p, 64, x, idx, w, q, s, sq, ss, poison=False)
    assert torch.equal(a, b)
    d = [t.to(DEV) for t in (x, idx, w, q, s, sq, ss)]
    out = torch.full((60, 384), 7.0, dtype=BF, device=DEV)
    moe.moe_experts_w4(p, 64, *d, out, moe.alloc_workspace(p, moe.MOE_CALL_EXPERTS_W4))
    assert torch.equal(out[:50], a) and (out[50:] == 7.0).all()


@pytest.mark.parametrize("T", [1, 64, 300])
def test_forward_routes_as_the_layer_does(T):
    c = MoEConfig("w4", T=T, H=256, E=16, top_k=4, I=256, num_shared=1, dtype=BF, x_std=1.0,
                  w_std=0.05, routed_scale=2.827, clip_limit=10.0)
    inp = make_inputs(c, seed=3, device=DEV)
    p = moe.MoEProblem.from_config(c)
    q, s = encode(p, inp["expert_w"], 64)
    sq, ss = encode(p, inp["shared_w"].unsqueeze(0), 64)
    ws = moe.alloc_workspace(p, moe.MOE_CALL_FORWARD_W4)
    ws[256:] = 0xff
    out = torch.full((T, c.H), float("nan"), dtype=BF, device=DEV)
    idx = torch.empty(T, 4, dtype=torch.int32, device=DEV)
    w = torch.empty(T, 4, device=DEV)
    moe.moe_forward_w4(p, 64, inp["x"], inp["gate_w"], None, q, s, sq, ss, out, idx, w, ws)
    torch.cuda.synchronize()
    assert moe.moe_read_device_status(ws) == 0
    cpu = to_cpu_inputs(inp)
    r = oracle.route(cpu["x"], cpu["gate_w"], 4, c.routed_scale)
    check_routing(idx.cpu().numpy(), w.cpu().numpy(), r, 4)
    # the layer on the GPU's own routing
    assert torch.equal(out, run_experts(p, 64, inp["x"], idx, w, q, s, sq, ss))
    want, bound = ref.w4_layer(cpu["x"][:64], idx.cpu()[:64], w.cpu()[:64],
                               ref.w4_weights(q, s, c.I, c.H, 64),
                               ref.w4_weights(sq, ss, c.I, c.H, 64)[0], 10.0, 64)
    ref.assert_within(out[:64], want, bound, "out")
    # idx and w may be left out
    out2 = torch.empty_like(out)
    moe.moe_forward_w4(p, 64, inp["x"], inp["gate_w"], None, q, s, sq, ss, out2, None, None, ws)
    assert torch.equal(out2, out)


def test_empty_batch():
    p = problem(0, 128, 4, 128, 2)
    q, s = draw_packed(4, p, 128, 23)
    e = torch.empty(0, 128, dtype=BF)
    run_experts(p, 128, e, torch.empty(0, 2, dtype=torch.int32), torch.empty(0, 2), q, s, None,
                None)
