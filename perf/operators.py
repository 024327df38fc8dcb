"""Cases and plain forms of the operators around the sparse MoE layer.

  norm   residual addition + root-mean-square norm, with E4M3 codes of the normed rows, and its
         backward pass (what feeds the layer's router, its bf16 and its FP8 forward)
  loss   the router's balance loss over packed sequences with its per-expert counts, and its
         gradient with respect to the router logits
  w4     the experts' products with 4-bit weights and group scales: dispatch, gate/up + SwiGLU,
         down, weighted combine, shared expert

With own = False ``run`` computes an operator from elementary torch operations in fp32; with
own = True it makes the library's calls.  ``exact`` computes it in fp64.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a decoding request through the pre-norm, bf16 stream (launch latency)
        dict(name="norm_one_token", op="norm", T=1, H=7168, dtype="bf16", residual=True, codes=False),
        # the prefill batch's pre-norm with the E4M3 rows for the FP8 layer
        dict(name="norm_prefill_codes", op="norm", T=4096, H=6144, dtype="bf16", residual=True,
             codes=True),
        # backward of the prefill-sized training batch, gradient of the residual stream joined in
        dict(name="norm_backward", op="norm_backward", T=4096, H=6144, dtype="bf16", residual=True),
        # fp32 training of a small model, odd batch, first block (no residual gradient)
        dict(name="norm_backward_fp32", op="norm_backward", T=333, H=1984, dtype="fp32",
             residual=False),
        # a decode-sized batch's balance statistics, one sequence
        dict(name="loss_small", op="loss", T=64, E=256, k=8, n_seq=1, masked=False, skew=False),
        # packed ragged training batch with padding and a skewed router
        dict(name="loss_packed", op="loss", T=16384, E=256, k=8, n_seq=37, masked=True, skew=True),
        # gradient for a large packed batch
        dict(name="loss_backward_packed", op="loss_backward", T=65536, E=256, k=8, n_seq=37,
             masked=True, skew=True),
        # gradient for the 32-expert top-2 router
        dict(name="loss_backward_e32", op="loss_backward", T=2048, E=32, k=2, n_seq=1,
             masked=False, skew=False),
        # one decoding request, 256 experts top-8 + shared
        dict(name="w4_one_token", op="w4", T=1, H=6144, E=256, I=2048, k=8, shared=1, clip=10.0,
             group=128),
        # the decode batch: most experts touched, about two rows each
        dict(name="w4_decode", op="w4", T=64, H=6144, E=256, I=2048, k=8, shared=1, clip=10.0,
             group=128),
        # odd batch on the 32-expert top-2 layer without shared expert or clamp, fine groups
        dict(name="w4_e32_groups32", op="w4", T=37, H=7168, E=32, I=2048, k=2, shared=0, clip=0.0,
             group=32),
        # the largest serving batch: about eight rows per expert
        dict(name="w4_large_batch", op="w4", T=256, H=6144, E=256, I=2048, k=8, shared=1,
             clip=10.0, group=64),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "loss", "loss_backward", "w4"])
    if op in ("norm", "norm_backward"):
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        c = dict(op=op, T=_log_int(rng, 1, 8192), H=64 * _log_int(rng, 1, 120), dtype=dtype,
                 residual=rng.random() < 0.7)
        if op == "norm":
            c["codes"] = dtype == "bf16" and rng.random() < 0.5
        return c
    if op in ("loss", "loss_backward"):
        E = _log_int(rng, 2, 256)
        return dict(op=op, T=_log_int(rng, 1, 65536), E=E, k=rng.randint(1, min(E, 8)),
                    n_seq=_log_int(rng, 1, 64), masked=rng.random() < 0.5,
                    skew=rng.random() < 0.5)
    E = _log_int(rng, 4, 128)
    return dict(op=op, T=_log_int(rng, 1, 256), H=128 * _log_int(rng, 1, 56), E=E,
                I=128 * _log_int(rng, 1, 16), k=rng.randint(1, min(E, 8)), shared=rng.randint(0, 1),
                clip=rng.choice([10.0, 0.0]), group=rng.choice([32, 64, 128]))


# ------------------------------------------------------------------ inputs

def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _sequences(c, seed):
    """Offsets of n_seq ragged sequences over T tokens: one of them empty and a few tokens behind
    the last where the batch is large enough (padding at the end of a packed batch)."""
    T, n = c["T"], c["n_seq"]
    if n == 1:
        return [0, T]
    r = random.Random(seed)
    end = T - T // 64
    cuts = sorted(r.randint(0, end) for _ in range(n - 1))
    cuts[len(cuts) // 2] = cuts[len(cuts) // 2 - 1] if len(cuts) > 1 else cuts[0]
    return [0] + cuts + [end]


def _prepare_loss(c, g, seed):
    T, E, k = c["T"], c["E"], c["k"]
    s = {"logits": torch.randn(T, E, generator=g, device="cuda") * 0.5}
    s["bias"] = None
    if c["skew"]:
        s["bias"] = -0.6 * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    s["idx"] = torch.topk(s["logits"] + (0.0 if s["bias"] is None else s["bias"]), k,
                          dim=-1).indices.to(torch.int32).contiguous()
    s["mask"] = None
    if c["masked"]:
        s["mask"] = (torch.rand(T, generator=g, device="cuda") < 0.9).to(torch.uint8)
    s["offsets"] = torch.tensor(_sequences(c, seed), dtype=torch.int32, device="cuda")
    n = c["n_seq"]
    s["loss"] = torch.empty(1, device="cuda")
    s["counts"] = torch.empty(n, E, dtype=torch.int32, device="cuda")
    s["tokens"] = torch.empty(n + 1, dtype=torch.int32, device="cuda")
    s["prob"] = torch.empty(n, E, device="cuda")
    if c["op"] == "loss_backward":
        # what the forward call left for it
        seq, live = _seq_of(s, T, n)
        s["counts"], s["tokens"] = _counts(s, c, seq, live)
        s["grad"] = torch.rand(1, generator=g, device="cuda") * 0.01 + 0.001
        s["dlogits"] = torch.empty(T, E, device="cuda")
    return s


def _prepare_w4(c, g):
    T, H, E, I, k, G = c["T"], c["H"], c["E"], c["I"], c["k"], c["group"]
    std = 0.006
    # 4-bit codes with the frequencies that normally distributed weights of a group scaled by its
    # largest magnitude have; the codes are independent, so any order of them is as good
    z = torch.distributions.Normal(0.0, 1.0).icdf((torch.arange(256, dtype=torch.float64) + 0.5)
                                                  / 256)
    nib = (torch.round(z * (7.0 / 2.6)).clamp(-7, 7) + 8).to(torch.int32)
    pair = (nib[:, None] + 16 * nib[None, :]).reshape(-1).to(torch.uint8).cuda()

    def weights(n):
        per = 3 * I * H // 2
        q = torch.empty(n, per, dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 26) // per)
        for e in range(0, n, step):
            part = q[e:e + step]
            part.copy_(pair[torch.randint(0, 65536, part.shape, generator=g, device="cuda",
                                          dtype=torch.int32)])
        sc = (std / 7.0) * (2.2 + 0.8 * torch.rand(n, 3 * I * H // G, generator=g, device="cuda"))
        return q, sc.to(torch.bfloat16)

    s = {"x": torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)}
    s["q"], s["sc"] = weights(E)
    s["sq"], s["ssc"] = weights(1) if c["shared"] else (None, None)
    logits = torch.randn(T, E, generator=g, device="cuda") * 0.5
    top, idx = torch.topk(logits, k, dim=-1)
    s["idx"] = idx.to(torch.int32).contiguous()
    s["w"] = (2.827 * torch.softmax(top, dim=-1)).contiguous()
    s["most"] = int(torch.bincount(idx.reshape(-1), minlength=E).max())  # rows of the fullest expert
    s["out"] = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    return s


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    if c["op"] in ("loss", "loss_backward"):
        s = _prepare_loss(c, g, seed)
    elif c["op"] == "w4":
        s = _prepare_w4(c, g)
    else:
        T, H, dt = c["T"], c["H"], _dtype(c)

        def rows(std=1.0):
            return (torch.randn(T, H, generator=g, device="cuda") * std).to(dt)

        w = (1.0 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(dt)
        if c["op"] == "norm":
            s = {"x": rows(), "res": rows(3.0) if c["residual"] else None, "weight": w,
                 "y": torch.empty(T, H, dtype=dt, device="cuda"),
                 "res_out": torch.empty(T, H, dtype=dt, device="cuda") if c["residual"] else None,
                 "y_q": None, "y_s": None}
            if c["codes"]:
                s["y_q"] = torch.empty(T, H, dtype=torch.uint8, device="cuda")
                s["y_s"] = torch.empty(T, device="cuda")
        else:
            s = {"dy": rows(0.01), "dres": rows(0.01) if c["residual"] else None, "h": rows(3.0),
                 "weight": w, "dx": torch.empty(T, H, dtype=dt, device="cuda"),
                 "dw": torch.empty(H, device="cuda")}
    s["case"] = c
    return s


# ------------------------------------------------------------------ plain forms (fp32)

def _pow2_scale(amax):
    """2^n with the smallest n for which 448 * 2^n >= amax; 1 where amax is 0."""
    m, e = torch.frexp(amax)
    n = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    s = torch.ldexp(torch.ones_like(amax), n)
    return torch.where(amax > 0, s, torch.ones_like(s))


def _norm_plain(s):
    x = s["x"].float()
    if s["res"] is not None:
        x = x + s["res"].float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    out = {"y": y.to(s["x"].dtype)}
    if s["res"] is not None:
        out["residual"] = x.to(s["x"].dtype)
    if s["y_q"] is not None:
        yr = out["y"].float()
        sc = _pow2_scale(yr.abs().amax(-1))
        out["codes"] = (yr / sc[:, None]).to(torch.float8_e4m3fn)
        out["scale"] = sc
    return out


def _norm_backward_plain(s):
    dy, h, w = s["dy"].float(), s["h"].float(), s["weight"].float()
    r = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    n = h * r
    gr = dy * w
    dx = r * (gr - n * (gr * n).mean(-1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(s["dy"].dtype), "dweight": (dy * n).sum(0)}


def _seq_of(s, T, n):
    """Sequence of each token (0 where it has none) and whether the token counts."""
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["offsets"], t, right=True) - 1
    live = (seq >= 0) & (seq < n)
    if s["mask"] is not None:
        live = live & (s["mask"] != 0)
    return seq.clamp(0, n - 1), live


def _counts(s, c, seq, live):
    n, E, k = c["n_seq"], c["E"], c["k"]
    at = seq[:, None] * E + s["idx"]
    counts = torch.zeros(n * E, dtype=torch.int32, device="cuda")
    counts.scatter_add_(0, at.reshape(-1), live[:, None].expand(-1, k).reshape(-1).int())
    tokens = torch.zeros(n, dtype=torch.int32, device="cuda")
    tokens.scatter_add_(0, seq, live.int())
    return counts.view(n, E), torch.cat([tokens, (tokens > 0).sum(dim=0, keepdim=True).int()])


def _probs(s):
    l = s["logits"] if s["bias"] is None else s["logits"] + s["bias"]
    ex = torch.exp(l - l.amax(-1, keepdim=True))
    return ex / ex.sum(-1, keepdim=True)


def _loss_plain(s):
    c = s["case"]
    n, E, k = c["n_seq"], c["E"], c["k"]
    seq, live = _seq_of(s, c["T"], n)
    counts, tokens = _counts(s, c, seq, live)
    p = _probs(s) * live[:, None]
    per = tokens[:n].float().clamp(min=1.0)[:, None]
    prob = torch.zeros(n, E, device="cuda").index_add_(0, seq, p) / per
    f = counts.float() / (per * k)
    loss = (E * (prob * f).sum() / tokens[n].float().clamp(min=1.0)).reshape(1)
    return {"loss": loss, "counts": counts, "tokens": tokens, "prob": prob}


def _loss_backward_plain(s):
    c = s["case"]
    n, E, k = c["n_seq"], c["E"], c["k"]
    seq, live = _seq_of(s, c["T"], n)
    per = s["tokens"][:n].float().clamp(min=1.0)
    f = s["counts"].float() / (per[:, None] * k)
    a = s["grad"] * E / (s["tokens"][n].float().clamp(min=1.0) * per)
    p = _probs(s)
    ft = f[seq]
    d = p * (ft - (p * ft).sum(-1, keepdim=True)) * a[seq][:, None]
    return {"dlogits": d * live[:, None]}


def _unpack_w4(q, sc, tiles, blocks, group):
    """Packed codes [n, tiles*blocks*2048] and scales -> fp32 [n, tiles, 2, 16, 128*blocks]."""
    n = q.shape[0]
    # [n, tile, block, half, k64, r, c, k32, k4, khi, k2]; the low nibble is row r, the high r + 8
    u = q.view(n, tiles, blocks, 2, 2, 8, 4, 2, 2, 2, 2)
    v = torch.stack([u & 15, u >> 4], dim=-1)
    v = v.permute(0, 1, 3, 11, 5, 2, 4, 7, 6, 8, 10, 9).reshape(n, tiles, 2, 16, 128 * blocks)
    w = v.float().sub_(8.0)
    sub = 128 // group
    t = sc.view(n, tiles, blocks, 8, sub, 2, 2).permute(0, 1, 5, 6, 3, 2, 4)
    t = t.reshape(n, tiles, 2, 16, blocks * sub, 1).float()
    return w.view(n, tiles, 2, 16, blocks * sub, group).mul_(t).view(n, tiles, 2, 16, 128 * blocks)


def _ffn_plain(x, q, sc, c):
    """x [n, rows, H] through expert n's SwiGLU FFN."""
    n, H, I, G = q.shape[0], c["H"], c["I"], c["group"]
    gu = I * H
    a = _unpack_w4(q[:, :gu], sc[:, :2 * I * H // G], I // 16, H // 128, G)
    a = torch.matmul(x, a.view(n, I // 16 * 32, H).transpose(1, 2)).view(n, -1, I // 16, 2, 16)
    gate, up = a[:, :, :, 0].reshape(n, -1, I), a[:, :, :, 1].reshape(n, -1, I)
    if c["clip"] > 0:
        gate, up = gate.clamp(-c["clip"], c["clip"]), up.clamp(-c["clip"], c["clip"])
    h = gate / (1.0 + torch.exp(-gate)) * up
    b = _unpack_w4(q[:, gu:], sc[:, 2 * I * H // G:], H // 32, I // 128, G)
    return torch.matmul(h, b.view(n, H, I).transpose(1, 2))


def _w4_plain(s):
    c = s["case"]
    T, H, E, k = c["T"], c["H"], c["E"], c["k"]
    x, idx = s["x"].float(), s["idx"].long()
    if T * k < E:
        # few assignments: only the experts that they name
        e = idx.reshape(-1)
        rows = x.repeat_interleave(k, 0)[:, None]
        y = _ffn_plain(rows, s["q"][e], s["sc"][e], c).view(T, k, H)
    else:
        # every expert, its rows padded to those of the fullest
        flat = idx.reshape(-1)
        order = torch.argsort(flat, stable=True)
        first = torch.searchsorted(flat[order], torch.arange(E, device="cuda"))
        place = torch.empty_like(flat)
        place[order] = torch.arange(T * k, device="cuda") - first[flat[order]]
        rows = torch.zeros(E, s["most"], H, device="cuda")
        rows[flat, place] = x.repeat_interleave(k, 0)
        y = _ffn_plain(rows, s["q"], s["sc"], c)[flat, place].view(T, k, H)
    out = (y * s["w"][:, :, None]).sum(1)
    if s["sq"] is not None:
        out = out + _ffn_plain(x[None], s["sq"], s["ssc"], c)[0]
    return {"out": out.to(torch.bfloat16)}


# ------------------------------------------------------------------ the library's calls

def _handle(s):
    """The problem and the workspace that a program keeps beside its buffers."""
    if "handle" not in s:
        from sparse_moe_layer_06_b200 import moe
        c = s["case"]
        p = moe.MoEProblem(T=c["T"], H=c.get("H", 64), E=c.get("E", 1), I=c.get("I", 64),
                           top_k=c.get("k", 1), num_shared=c.get("shared", 0), routed_scale=2.827,
                           clip_limit=c.get("clip", 0.0),
                           dtype=torch.float32 if c.get("dtype") == "fp32" else torch.bfloat16)
        ws = None
        if c["op"] == "norm_backward":
            ws = moe.alloc_workspace(p, moe.MOE_CALL_ADD_RMSNORM_BACKWARD)
        elif c["op"] == "loss":
            ws = moe.alloc_balance_workspace(p, c["n_seq"])
        elif c["op"] == "w4":
            ws = moe.alloc_workspace(p, moe.MOE_CALL_EXPERTS_W4)
            # a program lays its weights out once, when it loads them
            s["codes"] = _lay_out(s["q"]), None if s["sq"] is None else _lay_out(s["sq"])
        s["handle"] = (moe, p, ws)
    return s["handle"]


def _lay_out(q):
    """The codes in the library's order, a lane's 32 bytes of a block's half in one place:
    [.., k64, lane, 16 bytes] -> [.., lane, k64, 16 bytes]."""
    n = q.shape[0]
    return q.view(torch.int64).view(n, -1, 2, 32, 2).transpose(2, 3).reshape(n, -1).view(torch.uint8)


def _norm_own(s):
    moe, p, _ = _handle(s)
    moe.moe_add_rmsnorm(p, s["x"], s["res"], s["weight"], EPS, s["res_out"], s["y"], s["y_q"],
                        s["y_s"])
    out = {"y": s["y"]}
    if s["res"] is not None:
        out["residual"] = s["res_out"]
    if s["y_q"] is not None:
        out["codes"] = s["y_q"].view(torch.float8_e4m3fn)
        out["scale"] = s["y_s"]
    return out


def _norm_backward_own(s):
    moe, p, ws = _handle(s)
    moe.moe_add_rmsnorm_backward(p, s["dy"], s["dres"], s["h"], s["weight"], EPS, s["dx"], s["dw"],
                                 ws)
    return {"dx": s["dx"], "dweight": s["dw"]}


def _loss_own(s):
    moe, p, ws = _handle(s)
    moe.moe_balance_loss(p, s["logits"], s["bias"], s["idx"], s["mask"], s["offsets"], s["loss"],
                         s["counts"], s["tokens"], s["prob"], ws)
    return {"loss": s["loss"], "counts": s["counts"], "tokens": s["tokens"], "prob": s["prob"]}


def _loss_backward_own(s):
    moe, p, _ = _handle(s)
    moe.moe_balance_loss_backward(p, s["logits"], s["bias"], s["mask"], s["offsets"], s["counts"],
                                  s["tokens"], s["grad"], s["dlogits"])
    return {"dlogits": s["dlogits"]}


def _w4_own(s):
    moe, p, ws = _handle(s)
    q, sq = s["codes"]
    moe.moe_experts_w4(p, s["case"]["group"], s["x"], s["idx"], s["w"], q, s["sc"], sq, s["ssc"],
                       s["out"], ws)
    return {"out": s["out"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _norm_own, "norm_backward": _norm_backward_own, "loss": _loss_own,
                "loss_backward": _loss_backward_own, "w4": _w4_own}[op](state)
    return {"norm": _norm_plain, "norm_backward": _norm_backward_plain, "loss": _loss_plain,
            "loss_backward": _loss_backward_plain, "w4": _w4_plain}[op](state)


# ------------------------------------------------------------------ work

def work(case):
    c = case
    if c["op"] in ("norm", "norm_backward"):
        b = 2 if c["dtype"] == "bf16" else 4
        n = c["T"] * c["H"]
        if c["op"] == "norm":
            by = n * b * (4 if c["residual"] else 2) + c["H"] * b
            if c["codes"]:
                by += n + 4 * c["T"]
            return {"bytes": by, "flops": 6 * n}
        return {"bytes": n * b * (4 if c["residual"] else 3) + c["H"] * (b + 4), "flops": 12 * n}
    if c["op"] in ("loss", "loss_backward"):
        n = c["T"] * c["E"]
        small = c["T"] * (1 if c["masked"] else 0) + c["n_seq"] * c["E"] * 4
        if c["op"] == "loss":
            return {"bytes": 4 * n + 4 * c["T"] * c["k"] + small + c["n_seq"] * c["E"] * 4,
                    "flops": 6 * n}
        return {"bytes": 8 * n + small, "flops": 9 * n}
    E, k, T, S = c["E"], c["k"], c["T"], c["shared"]
    touched = E * (1.0 - (1.0 - k / E) ** T) + S
    weights = 3 * c["I"] * c["H"]
    return {"bytes": touched * weights * (0.5 + 2.0 / c["group"]) + T * c["H"] * 4 + T * k * 8,
            "flops": 2 * weights * T * (k + S)}


# ------------------------------------------------------------------ exact (fp64)

def _exact_norm(s):
    x = s["x"].double()
    if s["res"] is not None:
        x = x + s["res"].double()
    ms = torch.einsum("th,th->t", x, x) / x.shape[1]
    y = x / torch.sqrt(ms + EPS)[:, None] * s["weight"].double()
    out = {"y": y}
    if s["res"] is not None:
        out["residual"] = x
    if s["y_q"] is not None:
        sc = torch.exp2(torch.ceil(torch.log2(y.to(torch.bfloat16).abs().amax(-1).double()
                                              / E4M3_MAX)))
        out["codes"] = y / sc[:, None]
        out["scale"] = sc
    return out


def _exact_norm_backward(s):
    dy, h, w = s["dy"].double(), s["h"].double(), s["weight"].double()
    H = h.shape[1]
    ms = torch.einsum("th,th->t", h, h) / H + EPS
    dot = torch.einsum("th,th,h->t", dy, h, w)
    # d/dh_i of sum_j dy_j w_j h_j ms^-1/2
    dx = dy * w / torch.sqrt(ms)[:, None] - h * (dot / (H * ms * torch.sqrt(ms)))[:, None]
    if s["dres"] is not None:
        dx = dx + s["dres"].double()
    return {"dx": dx, "dweight": torch.einsum("th,th,t->h", dy, h, 1.0 / torch.sqrt(ms))}


def _exact_loss(s):
    c = s["case"]
    T, E, k, n = c["T"], c["E"], c["k"], c["n_seq"]
    off = s["offsets"].tolist()
    l = s["logits"].double() + (0.0 if s["bias"] is None else s["bias"].double())
    p = torch.softmax(l, dim=-1)
    live = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"].bool()
    chosen = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    chosen.scatter_(1, s["idx"].long(), 1.0)
    prob = torch.zeros(n, E, dtype=torch.float64, device="cuda")
    grad = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    used = sum(int(live[off[i]:off[i + 1]].any()) for i in range(n))
    loss = torch.zeros((), dtype=torch.float64, device="cuda")
    for i in range(n):
        sel = torch.nonzero(live[off[i]:off[i + 1]])[:, 0] + off[i]
        if sel.numel() == 0:
            continue
        prob[i] = p[sel].mean(0)
        f = chosen[sel].mean(0) / k
        loss = loss + E * torch.dot(prob[i], f) / used
        if c["op"] == "loss_backward":
            # J^T of the softmax applied to the loss's gradient with respect to p
            up = f * (E / used / sel.numel()) * s["grad"].double()
            ps = p[sel]
            grad[sel] = ps * up - ps * (ps @ up)[:, None]
    if c["op"] == "loss_backward":
        return {"dlogits": grad}
    return {"loss": loss.reshape(1), "counts": None, "tokens": None, "prob": prob}


def _exact_weights(q, sc, row0, rows, K, group, base_q, base_s, pair_rows):
    """Decoded fp64 [rows, K] of one matrix whose row i is row (i % pair_rows) + row0 of pair tile
    i // pair_rows, by the address of each weight."""
    i = torch.arange(rows, device="cuda")[:, None]
    kk = torch.arange(K, device="cuda")[None, :]
    tile, r = i // pair_rows, i % pair_rows + row0
    half, r16, blk, k = r // 16, r % 16, kk // 128, kk % 128
    lane = (r16 % 8) * 4 + k % 32 // 8
    word = k % 64 // 32 * 2 + k % 8 // 4
    byte = k % 2 * 2 + k % 4 // 2
    at = ((tile * (K // 128) + blk) * 2 + half) * 1024 + k // 64 * 512 + lane * 16 + word * 4 + byte
    v = (q[base_q + at] >> (4 * (r16 // 8)).to(torch.uint8)) & 15
    sub = 128 // group
    sat = (((tile * (K // 128) + blk) * 8 + r16 % 8) * sub + k // group) * 4 + half * 2 + r16 // 8
    return (v.double() - 8.0) * sc[base_s + sat].double()


def _exact_w4(s):
    c = s["case"]
    T, H, E, I, G = c["T"], c["H"], c["E"], c["I"], c["group"]
    x, idx, w = s["x"].double(), s["idx"].cpu(), s["w"].double()
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in list(range(E)) + ([-1] if c["shared"] else []):
        if e < 0:
            q, sc = s["sq"][0], s["ssc"][0]
            tok, wt = torch.arange(T), torch.ones(T, dtype=torch.float64, device="cuda")
        else:
            at = torch.nonzero(idx == e)
            if at.shape[0] == 0:
                continue
            q, sc, tok, slot = s["q"][e], s["sc"][e], at[:, 0], at[:, 1]
            wt = w[tok.cuda(), slot.cuda()]
        tok = tok.cuda()
        xe = x[tok]
        g = xe @ _exact_weights(q, sc, 0, I, H, G, 0, 0, 16).T
        u = xe @ _exact_weights(q, sc, 16, I, H, G, 0, 0, 16).T
        if c["clip"] > 0:
            g, u = g.clamp(-c["clip"], c["clip"]), u.clamp(-c["clip"], c["clip"])
        h = g * torch.sigmoid(g) * u
        y = h @ _exact_weights(q, sc, 0, H, I, G, I * H, 2 * I * H // G, 32).T
        out.index_add_(0, tok, y * wt[:, None])
    return {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    op = s["case"]["op"]
    if op == "norm":
        return _exact_norm(s)
    if op == "norm_backward":
        return _exact_norm_backward(s)
    if op == "w4":
        return _exact_w4(s)
    return _exact_loss(s)
