"""The operators together, as a serving step and a training step use them, and
captured into CUDA graphs."""
import pytest
import torch

import operator_reference as ref
from sparse_moe_layer_06_b200 import moe
from sparse_moe_layer_06_b200.workloads import MoEConfig, make_inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
CFG = MoEConfig("chain", T=96, H=256, E=16, top_k=4, I=256, num_shared=1, dtype=BF, x_std=1.0,
                w_std=0.05, routed_scale=2.827, clip_limit=10.0)


def setup(seed=5):
    inp = make_inputs(CFG, seed=seed, device=DEV)
    p = moe.MoEProblem.from_config(CFG)
    g = torch.Generator().manual_seed(seed)
    res = (torch.randn(CFG.T, CFG.H, generator=g) * 3).to(BF).to(DEV)
    w = (1 + 0.2 * torch.randn(CFG.H, generator=g)).to(BF).to(DEV)
    return inp, p, res, w


def empty(*shape, dtype=BF):
    return torch.empty(*shape, dtype=dtype, device=DEV)


def quantize_fp8(p, w):
    n = w.shape[0]
    q = empty(*w.shape, dtype=torch.uint8)
    s_gu, s_d = empty(n, 2, p.I, dtype=torch.float32), empty(n, p.H, dtype=torch.float32)
    moe.moe_quantize_weights_fp8(p, w, q, s_gu, s_d)
    return q, s_gu, s_d


def test_norm_codes_feed_the_fp8_layer():
    inp, p, res, w = setup()
    T, H = CFG.T, CFG.H
    y, ro, y_q, y_s = empty(T, H), empty(T, H), empty(T, H, dtype=torch.uint8), empty(
        T, dtype=torch.float32)
    moe.moe_add_rmsnorm(p, inp["x"], res, w, 1e-6, ro, y, y_q, y_s)
    weights = (*quantize_fp8(p, inp["expert_w"]), *quantize_fp8(p, inp["shared_w"].unsqueeze(0)))
    ws = moe.alloc_workspace(p, moe.MOE_CALL_FORWARD_FP8)
    a, b = empty(T, H), empty(T, H)
    moe.moe_forward_fp8(p, y, inp["gate_w"], None, *weights, a, None, None, ws)
    before = moe.moe_launch_count()
    moe.moe_forward_fp8_encoded(p, y, y_q, y_s, inp["gate_w"], None, *weights, b, None, None, ws)
    encoded = moe.moe_launch_count() - before
    moe.moe_forward_fp8(p, y, inp["gate_w"], None, *weights, a, None, None, ws)
    torch.cuda.synchronize()
    assert moe.moe_read_device_status(ws) == 0
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert moe.moe_launch_count() - before == 2 * encoded + 1  # the row encoder is not launched


def serving_step(inp, p, res, w, q4, bufs, ws):
    moe.moe_add_rmsnorm(p, inp["x"], res, w, 1e-6, bufs["ro"], bufs["y"])
    moe.moe_forward_w4(p, 128, bufs["y"], inp["gate_w"], None, *q4, bufs["out"], bufs["idx"],
                       bufs["w"], ws)
    # the next block's norm takes the layer's output and the residual stream
    moe.moe_add_rmsnorm(p, bufs["out"], bufs["ro"], w, 1e-6, bufs["ro2"], bufs["y2"])


def serving_setup(seed=5):
    inp, p, res, w = setup(seed)
    per = 3 * p.I * p.H
    q4 = []
    for wt in (inp["expert_w"], inp["shared_w"].unsqueeze(0)):
        q, s = empty(wt.shape[0], per // 2, dtype=torch.uint8), empty(wt.shape[0], per // 128)
        moe.moe_quantize_weights_w4(p, 128, wt, q, s)
        q4 += [q, s]
    bufs = {n: empty(CFG.T, CFG.H) for n in ("ro", "y", "out", "ro2", "y2")}
    bufs["idx"] = empty(CFG.T, CFG.top_k, dtype=torch.int32)
    bufs["w"] = empty(CFG.T, CFG.top_k, dtype=torch.float32)
    return inp, p, res, w, q4, bufs, moe.alloc_workspace(p, moe.MOE_CALL_FORWARD_W4)


def test_serving_step_matches_64_bits():
    inp, p, res, w, q4, bufs, ws = serving_setup()
    serving_step(inp, p, res, w, q4, bufs, ws)
    torch.cuda.synchronize()
    assert moe.moe_read_device_status(ws) == 0
    c = {n: t.cpu() for n, t in bufs.items()}
    _, y, _ = ref.norm(inp["x"].cpu(), res.cpu(), w.cpu(), 1e-6)
    ref.assert_within(c["y"], y, ref.norm_y_bound(y, BF), "y")
    n = 24
    want, bound = ref.w4_layer(c["y"][:n], c["idx"][:n], c["w"][:n],
                               ref.w4_weights(q4[0], q4[1], p.I, p.H, 128),
                               ref.w4_weights(q4[2], q4[3], p.I, p.H, 128)[0], 10.0, 128)
    ref.assert_within(c["out"][:n], want, bound, "out")
    _, y2, _ = ref.norm(c["out"], c["ro"], w.cpu(), 1e-6)
    ref.assert_within(c["y2"], y2, ref.norm_y_bound(y2, BF), "y2")


def training_step(inp, p, res, w, b, offsets, mask):
    moe.moe_add_rmsnorm(p, inp["x"], res, w, 1e-6, b["ro"], b["y"])
    moe.moe_router_logits(p, b["y"], inp["gate_w"], b["logits"], b["ws_l"])
    moe.moe_route(p, b["y"], inp["gate_w"], None, b["idx"], b["w"], b["ws_r"])
    moe.moe_balance_loss(p, b["logits"], None, b["idx"], mask, offsets, b["loss"], b["counts"],
                         b["tokens"], b["prob"], b["ws_b"])
    moe.moe_balance_loss_backward(p, b["logits"], None, mask, offsets, b["counts"], b["tokens"],
                                  b["one"], b["dlogits"])
    # the gate's own products are the caller's
    torch.matmul(b["dlogits"], inp["gate_w"].float(), out=b["dy32"])
    torch.matmul(b["dlogits"].T, b["y"].float(), out=b["dgate"])
    b["dy"].copy_(b["dy32"])
    moe.moe_add_rmsnorm_backward(p, b["dy"], None, b["ro"], w, 1e-6, b["dx"], b["dw"], b["ws_n"])


def training_buffers(p):
    T, H, E, k = CFG.T, CFG.H, CFG.E, CFG.top_k
    f = torch.float32
    b = {n: empty(T, H) for n in ("ro", "y", "dy", "dx")}
    b.update(logits=empty(T, E, dtype=f), idx=empty(T, k, dtype=torch.int32),
             w=empty(T, k, dtype=f), loss=empty(1, dtype=f),
             counts=empty(3, E, dtype=torch.int32), tokens=empty(4, dtype=torch.int32),
             prob=empty(3, E, dtype=f), dlogits=empty(T, E, dtype=f), dy32=empty(T, H, dtype=f),
             dgate=empty(E, H, dtype=f), dw=empty(H, dtype=f), one=torch.ones(1, device=DEV),
             ws_l=moe.alloc_workspace(p, moe.MOE_CALL_ROUTER_LOGITS),
             ws_r=moe.alloc_workspace(p, moe.MOE_CALL_ROUTE),
             ws_b=moe.alloc_balance_workspace(p, 3),
             ws_n=moe.alloc_workspace(p, moe.MOE_CALL_ADD_RMSNORM_BACKWARD))
    return b


def test_training_step_gradients_match_64_bits():
    inp, p, res, w = setup()
    b = training_buffers(p)
    offsets = torch.tensor([0, 40, 40, 90], dtype=torch.int32, device=DEV)
    mask = (torch.rand(CFG.T, generator=torch.Generator().manual_seed(1)) < 0.8).to(torch.uint8)
    training_step(inp, p, res, w, b, offsets, mask.to(DEV))
    torch.cuda.synchronize()
    c = {n: t.cpu() for n, t in b.items()}
    off = offsets.tolist()
    _, counts, tokens, _ = ref.balance_loss(c["logits"], None, c["idx"], mask, off, CFG.top_k)
    assert torch.equal(c["counts"], counts) and torch.equal(c["tokens"], tokens)
    d, mag = ref.balance_backward(c["logits"], None, mask, off, counts, tokens, 1.0, CFG.top_k)
    units = ref.prob_units(c["logits"], None)
    ref.assert_within(c["dlogits"], d, mag * (2 * units + 24) * 2.0 ** -24, "dlogits")
    dx, dw, mx, mw = ref.norm_backward(c["dy"], None, c["ro"], w.cpu(), 1e-6)
    ref.assert_within(c["dx"], dx, ref.norm_dx_bound(dx, mx, BF), "dx")
    ref.assert_within(c["dw"], dw, ref.norm_dw_bound(mw, CFG.T), "dweight")


@pytest.mark.parametrize("kind", ["serving", "training"])
def test_steps_replay_from_a_cuda_graph(kind):
    if kind == "serving":
        inp, p, res, w, q4, bufs, ws = serving_setup()
        step = lambda: serving_step(inp, p, res, w, q4, bufs, ws)  # noqa: E731
        names = ("out", "ro2", "y2", "idx")
    else:
        inp, p, res, w = setup()
        bufs = training_buffers(p)
        offsets = torch.tensor([0, 40, 40, 90], dtype=torch.int32, device=DEV)
        step = lambda: training_step(inp, p, res, w, bufs, offsets, None)  # noqa: E731
        names = ("loss", "counts", "tokens", "dlogits", "dx", "dw")
    step()
    torch.cuda.synchronize()
    eager = {n: bufs[n].clone() for n in names}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for n in names:
            bufs[n].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(bufs[n], eager[n]) for n in names)
    # a replay reads the inputs as they then are
    inp["x"].copy_(make_inputs(CFG, seed=77, device=DEV)["x"])
    graph.replay()
    torch.cuda.synchronize()
    got = {n: bufs[n].clone() for n in names}
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(bufs[n], got[n]) for n in names)
    del graph


def test_two_calls_at_once_on_two_streams():
    inp, p, res, w, q4, bufs, ws = serving_setup()
    serving_step(inp, p, res, w, q4, bufs, ws)
    torch.cuda.synchronize()
    want = bufs["y2"].clone()
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = [({n: torch.zeros_like(t) for n, t in bufs.items()},
             moe.alloc_workspace(p, moe.MOE_CALL_FORWARD_W4)) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, (b, wsp) in zip(streams, sets):
            with torch.cuda.stream(st):
                serving_step(inp, p, res, w, q4, b, wsp)
    torch.cuda.synchronize()
    assert all(torch.equal(b["y2"], want) for b, _ in sets)
