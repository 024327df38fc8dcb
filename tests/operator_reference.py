"""Plain 64-bit forms of the operators around the layer (norm, balance loss,
4-bit experts), written from their definitions, and the error bounds that the
GPU tests hold the kernels to.

Bounds.  A value rounded to a type of relative half step u (bf16 2^-8, fp32
2^-24) is off by at most u of itself; a chain of n fp32 additions by at most
n 2^-24 of the sum of the magnitudes added.  Each bound below is one rounding
to the output type plus the fp32 chain of that output, counted in units of
2^-24 and stated beside it.
"""
import numpy as np
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
F64 = torch.float64


def assert_within(got, want, bound, what):
    """|got - want| <= bound everywhere (all three broadcast, fp64)."""
    got, want = got.detach().cpu().to(F64), want.to(F64)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - want).abs() - bound
    assert (over <= 0).all(), (
        f"{what}: over its bound by {over.max().item():.3e} at {int(over.argmax())}, "
        f"max error {(got - want).abs().max().item():.3e}")


# ------------------------------------------------------------------ norm

def norm(x, res, w, eps):
    """s, y, r in fp64."""
    s = x.to(F64) + (0 if res is None else res.to(F64))
    r = (s.square().mean(-1, keepdim=True) + eps).rsqrt()
    return s, s * w.to(F64) * r, r


def norm_y_bound(y, dtype):
    # a thread adds at most 32 squares, 10 shuffle steps follow, each off by
    # 2^-24 of the (positive) sum, halved by the square root: 21; the mean, eps,
    # square root, quotient, s, s * w and the product with r: 7 more
    return y.abs() * (HALF_STEP[dtype] + 28 * 2.0 ** -24 * (1 + HALF_STEP[dtype]))


def norm_backward(dy, dres, h, w, eps):
    """dx, dweight and the magnitudes that their bounds count from."""
    dy, h, w = dy.to(F64), h.to(F64), w.to(F64)
    r = (h.square().mean(-1, keepdim=True) + eps).rsqrt()
    n, g = h * r, dy * w
    m = (g * n).mean(-1, keepdim=True)
    d = 0 if dres is None else dres.to(F64)
    dx = r * (g - n * m) + d
    mag = r * (g.abs() + n.abs() * (g * n).abs().mean(-1, keepdim=True)) + abs(d)
    return dx, (dy * n).sum(0), mag, (dy * n).abs().sum(0)


def norm_dx_bound(dx, mag, dtype):
    # the dot product's chain (32 terms of two products each, 10 shuffles: 44),
    # r (28, squared in the mean's factor: 56), the products and sums: 8
    return dx.abs() * HALF_STEP[dtype] + 110 * 2.0 ** -24 * mag * (1 + HALF_STEP[dtype])


def norm_dw_bound(mag, T):
    # r (28), two products; a CTA's rows (at most T/148 + 1), 37 partials (of at
    # most 1184) per warp, 32 warps
    return mag * (28 + 2 + T / 148 + 1 + 37 + 32) * 2.0 ** -24


# ------------------------------------------------------------------ balance loss

def spans(offsets, T):
    return [(0, T)] if offsets is None else list(zip(offsets[:-1], offsets[1:]))


def probs(logits, bias):
    l = logits.to(F64) + (0 if bias is None else bias.to(F64))
    mx = l.amax(-1, keepdim=True)
    mx = torch.where(torch.isinf(mx) & (mx < 0), torch.zeros_like(mx), mx)
    ex = torch.exp(l - mx)
    z = ex.sum(-1, keepdim=True)
    return torch.where(z > 0, ex / z, torch.zeros_like(ex))


def balance_loss(logits, bias, idx, mask, offsets, k):
    T, E = logits.shape
    p = probs(logits, bias)
    sp = spans(offsets, T)
    n_seq = len(sp)
    P = torch.zeros(n_seq, E, dtype=F64)
    counts = torch.zeros(n_seq, E, dtype=torch.int32)
    tokens = torch.zeros(n_seq + 1, dtype=torch.int32)
    loss = 0.0
    for s, (a, b) in enumerate(sp):
        live = [t for t in range(a, b) if mask is None or mask[t]]
        tokens[s] = len(live)
        for t in live:
            P[s] += p[t]
            for e in idx[t].tolist():
                if 0 <= e < E:
                    counts[s, e] += 1
        if live:
            P[s] /= len(live)
            loss += E * float((P[s] * counts[s].to(F64) / (len(live) * k)).sum())
    used = int((tokens[:-1] > 0).sum())
    tokens[-1] = used
    return loss / used if used else 0.0, counts, tokens, P


def balance_backward(logits, bias, mask, offsets, counts, tokens, grad, k):
    """dlogits and the magnitudes that its bound counts from."""
    T, E = logits.shape
    p = probs(logits, bias)
    d, mag = torch.zeros(T, E, dtype=F64), torch.zeros(T, E, dtype=F64)
    used = int(tokens[-1])
    for s, (a, b) in enumerate(spans(offsets, T)):
        n = int(tokens[s])
        if not n:
            continue
        f = counts[s].to(F64) / (n * k)
        for t in range(a, b):
            if mask is not None and not mask[t]:
                continue
            dot = (p[t] * f).sum()
            d[t] = grad * E / (used * n) * p[t] * (f - dot)
            mag[t] = abs(grad) * E / (used * n) * p[t] * (f + dot + 2.0 / E)
    return d, mag


def prob_units(logits, bias):
    """Error of a probability in units of 2^-24, with all |logit + bias| <= big.
    Numerator: the logit plus its bias (big), less the maximum (2 big), times
    log2 e as fp32 (product 2 big, constant 0.5 big, in units of the natural
    exponent) are absolute errors of the exponent; the approximate exponential is
    stated to 2^-22: 4.  The sum of numerators carries
    as much, and 13 additions; quotient and product: 2."""
    l = logits.to(F64) + (0 if bias is None else bias.to(F64))
    fin = l[torch.isfinite(l)]
    big = float(fin.abs().max()) if fin.numel() else 0.0
    return 2 * (5.5 * big + 4) + 15


# ------------------------------------------------------------------ 4-bit experts

def w4_encode(w, group):
    """Codes (0..15) and bf16-rounded scales of [..., K] weights, groups along K."""
    w32 = w.float().numpy()
    g = w32.reshape(*w32.shape[:-1], -1, group)
    amax = np.abs(g).max(-1)
    s = torch.from_numpy((amax / np.float32(7)).astype(np.float32)).to(torch.bfloat16).float()
    s = s.numpy()
    s = np.where(s == 0, np.float32(1), s)
    s = np.where(np.isfinite(g).all(-1), s, np.float32("nan"))
    with np.errstate(invalid="ignore"):
        # fp64 quotients of 24-bit by 8-bit values are never rounded onto a half
        c = np.rint(g.astype(np.float64) / s[..., None].astype(np.float64))
    c = np.where(np.isnan(c), 0, np.clip(c, -7, 7)).astype(np.int64) + 8
    return c.reshape(w32.shape), s


def _w4_matrix(q, sc, rows, K, group, pair_rows, first):
    """Decode one matrix of one expert by the address of each weight: row i is
    row first + i % pair_rows of pair tile i // pair_rows."""
    i, k = np.arange(rows)[:, None], np.arange(K)[None, :]
    tile, r = i // pair_rows, first + i % pair_rows
    half, r16, blk, kk = r // 16, r % 16, k // 128, k % 128
    b = kk // 32 * 8 + kk % 8 // 4 * 4 + kk % 2 * 2 + kk % 4 // 2
    lane = (r16 % 8) * 4 + kk % 32 // 8
    at = ((tile * (K // 128) + blk) * 2 + half) * 1024 + lane * 32 + b
    u = (q[at] >> (4 * (r16 // 8))) & 15
    sub = 128 // group
    sat = (((tile * (K // 128) + blk) * 8 + r16 % 8) * sub + kk // group) * 4 + half * 2 + r16 // 8
    return u, sc[sat]


def w4_unpack(q, sc, I, H, group):
    """One expert's packed bytes and scales (fp32) -> per matrix (codes, scales per weight)."""
    gu, gs = I * H, 2 * I * H // group
    gate = _w4_matrix(q[:gu], sc[:gs], I, H, group, 16, 0)
    up = _w4_matrix(q[:gu], sc[:gs], I, H, group, 16, 16)
    down = _w4_matrix(q[gu:], sc[gs:], H, I, group, 32, 0)
    return gate, up, down


def w4_weights(q, sc, I, H, group):
    """[n, ...] packed weights -> list of (gate [I,H], up [I,H], down [H,I]) in fp64."""
    out = []
    for e in range(q.shape[0]):
        m = w4_unpack(q[e].cpu().numpy().reshape(-1).astype(np.int64),
                      sc[e].float().cpu().numpy().reshape(-1), I, H, group)
        out.append(tuple(torch.from_numpy((u - 8) * s.astype(np.float64)) for u, s in m))
    return out


def w4_ffn(x, mats, clip, group):
    """FFN of rows x in fp64 and a bound on the kernel's error before the output rounding.

    The kernel takes a row's block of 128 values as 16-bit integers times a power
    of two a; the largest, amax, is 16191 a or more, so each value is off by at
    most a/2 <= 2^-14.9 amax.  Its sums over a group are exact integers; the
    two limbs are joined, scaled (two products) and added to the fp32 total, in
    K/group additions and 8 more over the warps: each of these steps is off by at
    most 2^-24 of the magnitudes added so far.  For chunks of up to four rows the
    limbs' sums stay apart and are joined at the end of K: as a value v a = (256 hi
    + lo) a has |lo| <= 128, the magnitudes are 256 |hi| a + |lo| a <= |v| a + 256 a,
    and 256 a <= amax 256/16191 < amax/63.  The clamp only shrinks errors;
    |silu'| <= 1.1; exp, sum and quotient: 2^-20 of h."""
    gate, up, down = mats
    H, I = gate.shape[1], gate.shape[0]

    def floor(v):  # 2^-14.9 of each block's largest magnitude
        return (v.abs().reshape(v.shape[0], -1, 128).amax(-1) * 2.0 ** -14.9
                ).repeat_interleave(128, -1)

    def product(v, dv, m):
        e = (m.shape[1] / group + 8 + 3) * 2.0 ** -24
        limbs = dv * (2.0 ** 14.9 / 63)
        return v @ m.T, dv @ m.abs().T + e * ((v.abs() + dv + limbs) @ m.abs().T)

    x = x.to(F64)
    g, dg = product(x, floor(x), gate)
    u, du = product(x, floor(x), up)
    if clip > 0:
        g, u = g.clamp(-clip, clip), u.clamp(-clip, clip)
    silu = g * torch.sigmoid(g)
    h = silu * u
    dh = 1.1 * dg * (u.abs() + du) + silu.abs() * du + 2.0 ** -20 * h.abs()
    dh = dh + 2.0 ** -24 * (h.abs() + dh) + floor(h.abs() + dh)
    return product(h, dh, down)


def w4_layer(x, idx, w, experts, shared, clip, group):
    """out in fp64 and the bound on a bf16 output."""
    T, H = x.shape
    out, err = torch.zeros(T, H, dtype=F64), torch.zeros(T, H, dtype=F64)
    mag = torch.zeros(T, H, dtype=F64)
    for t in range(T):
        for j in range(idx.shape[1]):
            e = int(idx[t, j])
            if not 0 <= e < len(experts):
                continue
            y, d = w4_ffn(x[t:t + 1], experts[e], clip, group)
            wt = float(w[t, j])
            out[t] += wt * y[0]
            err[t] += abs(wt) * d[0]
            mag[t] += abs(wt) * y[0].abs()
    if shared is not None:
        y, d = w4_ffn(x, shared, clip, group)
        out += y
        err += d
        mag += y.abs()
    # the weight's product and up to k + 1 additions in fp32, then the output's rounding
    err = err + (idx.shape[1] + 3) * 2.0 ** -24 * (mag + err)
    return out, out.abs() * 2.0 ** -8 + err * (1 + 2.0 ** -8)
