"""Balance loss over packed sequences and its gradient against the 64-bit forms
in operator_reference (which states the bounds)."""
import pytest
import torch

import operator_reference as ref
from sparse_moe_layer_06_b200 import moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


def problem(T, E, k):
    return moe.MoEProblem(T=T, H=64, E=E, I=64, top_k=k, num_shared=0, routed_scale=1.0,
                          clip_limit=0.0, dtype=torch.bfloat16)


def draw(T, E, k, seed, skew=0.0, masked=0.0):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, generator=g) * 1.5
    bias = -skew * torch.log(torch.arange(1, E + 1).float()) if skew else None
    idx = torch.topk(logits + (0 if bias is None else bias), k, dim=-1).indices.to(torch.int32)
    mask = (torch.rand(T, generator=g) >= masked).to(torch.uint8) if masked else None
    return logits, bias, idx, mask


def run_loss(logits, bias, idx, mask, offsets, status=0):
    T, E = logits.shape
    k, n = idx.shape[1], 1 if offsets is None else len(offsets) - 1
    p = problem(T, E, k)
    d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device=DEV)
    out = (torch.full((1,), float("nan"), device=DEV),
           torch.full((n, E), -5, dtype=torch.int32, device=DEV),
           torch.full((n + 1,), -5, dtype=torch.int32, device=DEV),
           torch.full((n, E), float("nan"), device=DEV))
    ws = moe.alloc_balance_workspace(p, n)
    ws[256:] = 0xff  # nothing of it is read before it is written
    moe.moe_balance_loss(p, d(logits), d(bias), d(idx), d(mask), off, *out, ws)
    torch.cuda.synchronize()
    assert moe.moe_read_device_status(ws) == status
    return out


def run_backward(logits, bias, mask, offsets, counts, tokens, grad, k):
    T, E = logits.shape
    d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device=DEV)
    dl = torch.full((T, E), float("nan"), device=DEV)
    moe.moe_balance_loss_backward(problem(T, E, k), d(logits), d(bias), d(mask), off, d(counts),
                                  d(tokens), torch.tensor([grad], device=DEV), dl)
    torch.cuda.synchronize()
    return dl


def check(logits, bias, idx, mask, offsets, grad=0.37):
    k = idx.shape[1]
    loss, counts, tokens, P = run_loss(logits, bias, idx, mask, offsets)
    rl, rc, rt, rP = ref.balance_loss(logits, bias, idx, mask, offsets, k)
    units = ref.prob_units(logits, bias)
    # a warp's tokens of a window and the 8 warps in fp32 (22 additions), the
    # windows in fp64, one rounding of the result
    assert torch.equal(counts.cpu(), rc) and torch.equal(tokens.cpu(), rt)
    ref.assert_within(P, rP, rP * (units + 24) * 2.0 ** -24, "mean_prob")
    assert abs(float(loss[0]) - rl) <= abs(rl) * (units + 26) * 2.0 ** -24
    dl = run_backward(logits, bias, mask, offsets, counts, tokens, grad, k)
    d, mag = ref.balance_backward(logits, bias, mask, offsets, rc, rt, grad, k)
    # the probability twice, the shares (3), 13 additions, 5 products
    ref.assert_within(dl, d, mag * (2 * units + 24) * 2.0 ** -24, "dlogits")
    return loss, counts, tokens, P, dl


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 2, 1), (1, 256, 8), (7, 5, 5), (8, 32, 2),
                                   (9, 33, 4), (64, 256, 8), (300, 100, 32), (1000, 256, 2)])
@pytest.mark.parametrize("skew,masked", [(0.0, 0.0), (0.6, 0.3)])
def test_one_sequence(T, E, k, skew, masked):
    check(*draw(T, E, k, 1, skew, masked), None)


@pytest.mark.parametrize("offsets", [
    [0, 0, 200], [0, 1, 2, 3, 200], [5, 60, 60, 60, 61, 150], [0, 8, 16, 24, 32], [200, 200],
    [0] + list(range(1, 200, 3)) + [200], [0, 7, 9, 200, 200, 200]])
@pytest.mark.parametrize("masked", [0.0, 0.4])
def test_packed_sequences(offsets, masked):
    check(*draw(200, 48, 3, 2, 0.6, masked), offsets)


def test_windows_that_end_inside_sequences():
    # 5000 tokens: windows of 16, sequences that start and end inside them, more
    # sequences than a window holds, an empty one on a window's border
    offsets = [3, 16, 16, 17, 30, 33, 1000, 1001, 1002, 1003, 1004, 4990]
    check(*draw(5000, 16, 2, 3, 0.6, 0.1), offsets)


def test_every_token_masked():
    logits, bias, idx, _ = draw(50, 16, 2, 4)
    mask = torch.zeros(50, dtype=torch.uint8)
    mask[45:] = 1
    check(logits, bias, idx, mask, [0, 20, 40])       # no token counts anywhere
    loss, _, tokens, _, dl = check(logits, bias, idx, mask, [0, 20, 50])
    assert tokens.tolist() == [0, 5, 1] and (dl[:45] == 0).all()


def test_masked_logits_of_minus_infinity_and_padding_garbage():
    logits, _, idx, _ = draw(40, 24, 2, 5)
    logits[:, 20:] = float("-inf")                    # experts that are masked off
    logits[7] = float("-inf")                         # a token with every expert masked off
    logits[8, :] = torch.finfo(torch.float32).min     # masked with the lowest value: uniform
    idx = torch.topk(logits, 2, dim=-1).indices.to(torch.int32)
    mask = torch.ones(40, dtype=torch.uint8)
    mask[30:] = 0
    logits[30:] = float("nan")                        # padding that is not read
    clean = logits.clone()
    clean[30:] = 0
    loss, counts, tokens, P = run_loss(logits, None, idx, mask, None)
    rl, rc, rt, rP = ref.balance_loss(clean, None, idx, mask, None, 2)
    assert torch.equal(counts.cpu(), rc) and torch.equal(tokens.cpu(), rt)
    units = ref.prob_units(torch.where(clean < -1e30, torch.zeros(()), clean), None)
    ref.assert_within(P, rP, rP * (units + 24) * 2.0 ** -24, "mean_prob")
    assert abs(float(loss[0]) - rl) <= abs(rl) * (units + 26) * 2.0 ** -24
    dl = run_backward(logits, None, mask, None, counts, tokens, 1.0, 2)
    d, mag = ref.balance_backward(clean, None, mask, None, rc, rt, 1.0, 2)
    ref.assert_within(dl, d, mag * (2 * units + 24) * 2.0 ** -24, "dlogits")
    assert (dl[7] == 0).all() and (dl[30:] == 0).all()


def test_gradient_against_differences():
    # the counts held, as the loss defines its gradient: central differences in
    # fp64 at d = 1e-4 are off by about 1e-9 of the loss
    logits, bias, idx, mask = draw(30, 12, 3, 6, 0.6, 0.2)
    offsets, d = [0, 4, 4, 26], 1e-4
    _, counts, tokens, _ = run_loss(logits, bias, idx, mask, offsets)
    dl = run_backward(logits, bias, mask, offsets, counts, tokens, 1.0, 3).cpu().to(ref.F64)
    g = torch.Generator().manual_seed(7)
    _, mag = ref.balance_backward(logits, bias, mask, offsets, counts.cpu(), tokens.cpu(), 1.0, 3)
    for _ in range(4):
        v = torch.randn(30, 12, generator=g, dtype=ref.F64)
        hi, lo = (ref.balance_loss(logits.to(ref.F64) + sgn * d * v, bias, idx, mask, offsets,
                                   3)[0] for sgn in (1, -1))
        bound = (mag * v.abs()).sum() * (2 * ref.prob_units(logits, bias) + 24) * 2.0 ** -24 + 1e-7
        assert abs((dl * v).sum() - (hi - lo) / (2 * d)) <= bound


def test_agrees_with_the_router_statistics():
    T, H, E, k = 333, 128, 32, 4
    p = moe.MoEProblem(T=T, H=H, E=E, I=64, top_k=k, num_shared=0, routed_scale=1.0,
                       clip_limit=0.0, dtype=torch.bfloat16)
    g = torch.Generator().manual_seed(8)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV)
    gate = (torch.randn(E, H, generator=g) * 0.1).to(torch.bfloat16).to(DEV)
    logits = torch.empty(T, E, device=DEV)
    idx = torch.empty(T, k, dtype=torch.int32, device=DEV)
    w = torch.empty(T, k, device=DEV)
    P, f, aux = (torch.empty(n, device=DEV) for n in (E, E, 1))
    moe.moe_router_logits(p, x, gate, logits, moe.alloc_workspace(p, moe.MOE_CALL_ROUTER_LOGITS))
    moe.moe_route(p, x, gate, None, idx, w, moe.alloc_workspace(p, moe.MOE_CALL_ROUTE))
    moe.moe_router_stats(p, x, gate, None, P, f, aux, None, None, 0.9,
                         moe.alloc_workspace(p, moe.MOE_CALL_ROUTER_STATS))
    loss, counts, tokens, mean = run_loss(logits.cpu(), None, idx.cpu(), None, None)
    # the two calls' logits differ in the order of their K sums
    torch.testing.assert_close(loss, aux, rtol=1e-5, atol=0)
    torch.testing.assert_close(mean[0], P, rtol=1e-5, atol=0)
    assert torch.equal(counts[0].cpu(), (f * T * k).round().int().cpu())


def test_bad_indexes_and_offsets_set_the_error_word():
    logits, _, idx, _ = draw(20, 8, 2, 9)
    bad = idx.clone()
    bad[3, 0], bad[4, 1] = -1, 8
    good = run_loss(logits, None, idx, None, None)
    loss, counts, tokens, P = run_loss(logits, None, bad, None, None,
                                       status=moe.MOE_ERR_BAD_INDEX)
    assert int(counts.sum()) == 38 and int(tokens[0]) == 20 and torch.equal(P, good[3])
    # a sequence that ends before it starts, and one that ends behind the batch
    _, counts, tokens, _ = run_loss(logits, None, idx, None, [5, 2, 10],
                                    status=moe.MOE_ERR_BAD_INDEX)
    assert tokens.tolist()[0] == 0
    _, counts, tokens, _ = run_loss(logits, None, idx, None, [0, 5, 21],
                                    status=moe.MOE_ERR_BAD_INDEX)
    assert tokens.tolist() == [5, 0, 1]


def test_reproducible_and_empty_batch():
    args = draw(3000, 64, 4, 10, 0.6, 0.2)
    a, b = run_loss(*args, [0, 100, 2990]), run_loss(*args, [0, 100, 2990])
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    e = torch.empty(0, 16), None, torch.empty(0, 2, dtype=torch.int32), None
    loss, counts, tokens, P = run_loss(*e, None)
    assert float(loss[0]) == 0 and (counts == 0).all() and tokens.tolist() == [0, 0]
    assert (P == 0).all()
    assert run_backward(e[0], None, None, None, counts, tokens, 1.0, 2).numel() == 0


def test_many_sequences():
    # more than 1024: three rounds of the search for a window's first sequence
    g = torch.Generator().manual_seed(11)
    cuts = torch.randint(0, 3001, (2500,), generator=g).sort().values.tolist()
    check(*draw(3000, 16, 2, 12, 0.6, 0.2), [0] + cuts + [3000])


def test_tokens_past_the_32_bit_offset():
    # the tokens of the last sequence lie behind element 2^31 of the logits; the
    # others are masked, so their (uninitialised) logits are not read
    T, E, k, n = (1 << 23) + 777, 256, 2, 900
    logits, bias, idx, _ = draw(n, E, k, 13, 0.6)
    lg = torch.empty(T, E, device=DEV)
    lg[T - n:] = logits.to(DEV)
    ix = torch.zeros(T, k, dtype=torch.int32, device=DEV)
    ix[T - n:] = idx.to(DEV)
    mask = torch.zeros(T, dtype=torch.uint8, device=DEV)
    mask[T - n:] = 1
    offsets = [0, 100, T - n, T]
    loss, counts, tokens, P = run_loss(lg, bias, ix, mask, offsets)
    rl, rc, rt, rP = ref.balance_loss(logits, bias, idx, None, None, k)
    units = ref.prob_units(logits, bias)
    assert torch.equal(counts[2].cpu(), rc[0]) and tokens.tolist() == [0, 0, n, 1]
    # (a warp's share of a window is over 2000 tokens here, so it adds up to n of them)
    ref.assert_within(P[2], rP[0], rP[0] * (units + n + 8) * 2.0 ** -24, "mean_prob")
    assert abs(float(loss[0]) - rl) <= abs(rl) * (units + n + 10) * 2.0 ** -24
    dl = run_backward(lg, bias, mask, offsets, counts, tokens, 0.37, k)
    d, mag = ref.balance_backward(logits, bias, None, None, rc, rt, 0.37, k)
    ref.assert_within(dl[T - n:], d, mag * (2 * units + 24) * 2.0 ** -24, "dlogits")
    assert not dl[:T - n].any()


@pytest.mark.parametrize("T", [1, 15, 64, 95, 96, 97])
@pytest.mark.parametrize("E,k", [(32, 2), (50, 3), (100, 4), (250, 8), (256, 8)])
def test_small_batches_of_one_sequence(T, E, k):
    # one launch up to 96 tokens: whole, inside offsets, empty, offsets out of range
    args = draw(T, E, k, 14, 0.6, 0.3)
    check(*args, None)
    check(*args, [T // 3, T - T // 4])
    check(*args, [T, T])
    before = moe.moe_launch_count()
    loss, counts, tokens, P = run_loss(*args, [0, T + 1], status=moe.MOE_ERR_BAD_INDEX)
    assert moe.moe_launch_count() - before == (1 if T <= 96 else 2)
    assert float(loss[0]) == 0 and tokens.tolist() == [0, 0] and not counts.any()
    assert not P.any()
    bad = args[2].clone()
    bad[0, 0] = E
    full = args[3].clone().fill_(1)
    _, counts, tokens, _ = run_loss(args[0], args[1], bad, full, None,
                                    status=moe.MOE_ERR_BAD_INDEX)
    assert int(counts.sum()) == T * k - 1 and tokens.tolist() == [T, 1]


# the experts of a sequence in four, two and one CTAs of pass 2, with the last one
# part full, and windows that many sequences share
@pytest.mark.parametrize("E", [33, 100, 130, 256])
@pytest.mark.parametrize("n_seq", [2, 37, 60, 100, 149])
def test_wide_routers_over_many_sequences(E, n_seq):
    g = torch.Generator().manual_seed(15)
    cuts = torch.randint(0, 601, (n_seq - 1,), generator=g).sort().values.tolist()
    check(*draw(600, E, 4, 16, 0.6, 0.2), [0] + cuts + [600])
