"""4-bit experts: chunks of every kind in one call (up to four rows, five to eight,
more than a chunk) for each form of the products, and the sizes that the path is for
against 64-bit forms computed on the GPU."""
import pytest
import torch

import operator_reference as ref
from sparse_moe_layer_06_b200 import moe
from test_gpu_w4 import draw_packed, problem, run_experts
from test_gpu_w4_rows import bounded, layer

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def routing(T, k, counts, seed=80):
    """Routing with these rows per expert; a token's experts are distinct."""
    flat = [e for e, n in enumerate(counts) for _ in range(n)]
    assert len(flat) == T * k and max(counts) <= T
    idx = torch.tensor([[flat[t + T * j] for j in range(k)] for t in range(T)], dtype=torch.int32)
    g = torch.Generator().manual_seed(seed)
    return idx[torch.randperm(T, generator=g)], torch.rand(T, k, generator=g) + 0.1


# mean rows up to 4.5 (one column tile of 8 rows) and above (two): experts with up to four
# rows, with five to eight, with more, without any
COUNTS = {
    "one": (24, 2, [9, 8, 1, 7, 6, 2, 5, 4, 3, 1, 1, 1, 0, 0, 0, 0]),
    "one, shared": (7, 2, [7, 0, 3, 2, 1, 1, 0, 0]),
    "one, many rows": (23, 2, [23, 0, 4, 5, 0, 7, 0, 1, 1, 1, 1, 1, 1, 1]),
    "two": (40, 2, [17, 16, 1, 9, 8, 12, 4, 13, 0, 0]),
    "two, shared": (33, 3, [33, 1, 32, 3, 16, 7, 4, 2, 1]),
}


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("name", COUNTS)
@pytest.mark.parametrize("outliers", [False, True])
def test_chunks_of_every_kind(name, group, outliers):
    T, k, counts = COUNTS[name]
    E, H, I = len(counts), 256, 2048
    few = T * k / E <= 4.5
    assert few == name.startswith("one")
    # 128 pair tiles for each chunk: the CTAs' runs go from one kind of chunk to another
    shared = int("shared" in name)
    sizes = counts + [T] * shared
    most = 8 if few else 16
    parts = [min(most, n - a) for n in sizes for a in range(0, n, most)]
    assert any(1 <= n <= 4 for n in parts) and any(5 <= n <= 8 for n in parts)
    assert few or any(n > 8 for n in parts)
    chunks = len(parts)
    assert chunks * (I // 16) > 148 * 4 and chunks * (I // 16) % 148
    p = problem(T, H, E, I, k, shared, 10.0)
    q, s = draw_packed(E, p, group, 81)
    sq, ss = draw_packed(1, p, group, 82) if shared else (None, None)
    idx, w = routing(T, k, counts)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(83))
    if outliers:
        x[::3, 9], x[1::3, 140] = 900.0, -2500.0
    x = x.to(BF)
    out = run_experts(p, group, x, idx, w, q, s, sq, ss)
    sh = ref.w4_weights(sq, ss, I, H, group)[0] if shared else None
    want, bound = layer(x, idx, w, ref.w4_weights(q, s, I, H, group), sh, 10.0, group)
    ref.assert_within(out, want, bound, "out")


# ------------------------------------------------------------------ full sizes

def decode(q, sc, rows, K, group, pair_rows, first):
    """One matrix in 64 bits on the GPU, by the address of each weight."""
    i, k = torch.arange(rows, device=DEV)[:, None], torch.arange(K, device=DEV)[None, :]
    tile, r = i // pair_rows, first + i % pair_rows
    half, r16, blk, kk = r // 16, r % 16, k // 128, k % 128
    b = kk // 32 * 8 + kk % 8 // 4 * 4 + kk % 2 * 2 + kk % 4 // 2
    at = ((tile * (K // 128) + blk) * 2 + half) * 1024 + ((r16 % 8) * 4 + kk % 32 // 8) * 32 + b
    u = (q[at] >> (4 * (r16 // 8)).to(torch.uint8)) & 15
    sub = 128 // group
    sat = (((tile * (K // 128) + blk) * 8 + r16 % 8) * sub + kk // group) * 4 + half * 2 + r16 // 8
    return (u.to(ref.F64) - 8) * sc[sat].to(ref.F64)


def matrices(q, sc, I, H, group):
    gu, gs = I * H, 2 * I * H // group
    return (decode(q, sc, I, H, group, 16, 0), decode(q, sc, I, H, group, 16, 16),
            decode(q[gu:], sc[gs:], H, I, group, 32, 0))


def test_decode_is_the_other_decode():
    p = problem(1, 256, 1, 384, 1)
    q, s = draw_packed(1, p, 64, 84)
    for a, b in zip(matrices(q[0].to(DEV), s[0].to(DEV), 384, 256, 64),
                    ref.w4_weights(q, s, 384, 256, 64)[0]):
        assert torch.equal(a.cpu(), b)


# the decode batch (about two rows an expert, one column tile); a batch of 32 rows an expert
# (two column tiles, chunks of 12 rows in gate/up); every token on the same eight experts
@pytest.mark.parametrize("T,E,group,skewed", [(64, 256, 128, False), (256, 64, 64, False),
                                              (64, 256, 32, True), (1, 256, 128, False)])
def test_full_size_layer(T, E, group, skewed):
    H, I, k = 6144, 2048, 8
    p = problem(T, H, E, I, k, 1, 10.0)
    g = torch.Generator(device=DEV).manual_seed(85)
    per = 3 * I * H

    def weights(n):
        q = torch.randint(0, 256, (n, per // 2), generator=g, dtype=torch.uint8, device=DEV)
        return q, (0.003 * (0.5 + torch.rand(n, per // group, generator=g, device=DEV))).to(BF)

    q, s = weights(E)
    sq, ss = weights(1)
    x = torch.randn(T, H, generator=g, device=DEV)
    x[::4, 1000], x[1::4, 5] = 1500.0, 600.0  # some rows have an outlier channel
    x = x.to(BF)
    logits = torch.randn(T, E, generator=g, device=DEV)
    if skewed:
        logits[:, 17:17 + k] += 100.0
    idx = logits.topk(k).indices.to(torch.int32)
    w = torch.rand(T, k, generator=g, device=DEV) + 0.1
    out = run_experts(p, group, x, idx, w, q, s, sq, ss)
    want, err, mag = (torch.zeros(T, H, dtype=ref.F64, device=DEV) for _ in range(3))
    for e in range(E + 1):
        if e < E:
            t, j = torch.nonzero(idx == e, as_tuple=True)
            wt = w[t, j].to(ref.F64)[:, None]
        else:
            t, wt = torch.arange(T, device=DEV), torch.ones(T, 1, dtype=ref.F64, device=DEV)
        if len(t):
            m = matrices(q[e], s[e], I, H, group) if e < E else matrices(sq[0], ss[0], I, H, group)
            y, d = bounded(x[t], m, 10.0, group)
            want.index_add_(0, t, wt * y)
            err.index_add_(0, t, wt * d)
            mag.index_add_(0, t, wt * y.abs())
    err = err + (k + 3) * 2.0 ** -24 * (mag + err)
    bound = want.abs() * 2.0 ** -8 + err * (1 + 2.0 ** -8)
    ref.assert_within(out, want.cpu(), bound.cpu(), "out")
    # the errors as a whole are those of the output's rounding, at most half a step
    rel = (out.to(ref.F64) - want).square().sum(-1).sqrt() / want.square().sum(-1).sqrt()
    assert rel.max() < 2.0 ** -8
