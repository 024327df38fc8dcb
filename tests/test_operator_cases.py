"""The timed cases' plain forms, their 64-bit forms and the library's calls say the
same: what the cases hand over (packed 4-bit codes above all) is what the calls read."""
import importlib.util
import os

import pytest
import torch

import operator_reference as ref

PATH = os.path.join(os.path.dirname(__file__), "..", "perf", "operators.py")


@pytest.fixture()
def ops():
    spec = importlib.util.spec_from_file_location("operator_cases", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("group", [32, 64, 128])
def test_laid_out_codes_are_the_plain_forms_weights(ops, group):
    n, H, I = 2, 384, 256
    g = torch.Generator().manual_seed(1)
    per = 3 * I * H
    q = torch.randint(0, 256, (n, per // 2), generator=g, dtype=torch.int32).to(torch.uint8)
    sc = torch.rand(n, per // group, generator=g).to(torch.bfloat16)
    gu, gs = I * H, 2 * I * H // group
    a = ops._unpack_w4(q[:, :gu], sc[:, :gs], I // 16, H // 128, group)
    d = ops._unpack_w4(q[:, gu:], sc[:, gs:], H // 32, I // 128, group).reshape(n, H, I)
    laid = ops._lay_out(q)
    assert laid.shape == q.shape and laid.is_contiguous()
    for e, (gate, up, down) in enumerate(ref.w4_weights(laid, sc, I, H, group)):
        # (u - 8) s in fp32 is exact: 4 bits times 8
        assert torch.equal(a[e, :, 0].reshape(I, H).to(ref.F64), gate)
        assert torch.equal(a[e, :, 1].reshape(I, H).to(ref.F64), up)
        assert torch.equal(d[e].to(ref.F64), down)


def both(ops, case, seed=3):
    """Outputs of the plain form, of the library's calls, and in 64 bits."""
    s = ops.prepare(case, seed)
    ops.own = False
    plain = {k: v.clone() for k, v in ops.run(s).items()}
    ops.own = True
    got = {k: v.clone() for k, v in ops.run(s).items()}
    torch.cuda.synchronize()
    return s, plain, got, ops.exact(case, seed)


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,shared,clip,group", [(1, 4, 2, 1, 10.0, 128), (5, 4, 2, 1, 0.0, 64),
                                                     (9, 16, 3, 0, 10.0, 32)])
def test_w4_calls_and_plain_form(ops, T, E, k, shared, clip, group):
    case = dict(op="w4", T=T, H=256, E=E, I=384, k=k, shared=shared, clip=clip, group=group)
    s, plain, got, exact = both(ops, case)
    sh = ref.w4_weights(ops._lay_out(s["sq"]), s["ssc"], 384, 256, group)[0] if shared else None
    want, bound = ref.w4_layer(s["x"].cpu(), s["idx"].cpu(), s["w"].cpu(),
                               ref.w4_weights(ops._lay_out(s["q"]), s["sc"], 384, 256, group), sh,
                               clip, group)
    # the two 64-bit forms differ by the order of their sums
    assert (exact["out"].cpu() - want).abs().max() <= 1e-12 * want.abs().max()
    ref.assert_within(got["out"], want, bound, "the calls")
    # fp32 chains of up to 384 terms: 2^-24 (384 + 12) < 2^-15 of the magnitudes, inside the
    # kernel's 2^-14.9 of a block's largest
    ref.assert_within(plain["out"], want, bound, "the plain form")


@pytest.mark.gpu
@pytest.mark.parametrize("masked", [False, True])
def test_loss_calls_and_plain_form(ops, masked):
    c = dict(T=300, E=48, k=3, n_seq=5, masked=masked, skew=True)
    s, plain, got, exact = both(ops, dict(op="loss", **c))
    units = ref.prob_units(s["logits"].cpu(), s["bias"].cpu())
    for out in (plain, got):
        assert torch.equal(out["counts"], plain["counts"])
        assert torch.equal(out["tokens"], plain["tokens"])
        # sums of up to 300 tokens in fp32, in whatever order
        P = exact["prob"].cpu()
        ref.assert_within(out["prob"], P, P * (units + 302) * 2.0 ** -24, "prob")
        L = float(exact["loss"])
        assert abs(float(out["loss"]) - L) <= L * (units + 302 + 5 * 48) * 2.0 ** -24
    s, plain, got, exact = both(ops, dict(op="loss_backward", **c))
    d = exact["dlogits"].cpu()
    off = None if s["offsets"] is None else s["offsets"].tolist()
    mask = None if s["mask"] is None else s["mask"].cpu()
    _, mag = ref.balance_backward(s["logits"].cpu(), s["bias"].cpu(), mask, off,
                                  s["counts"].cpu(), s["tokens"].cpu(), float(s["grad"]), 3)
    for out in (plain, got):
        # the dot product of the plain form: up to 48 additions
        ref.assert_within(out["dlogits"], d, mag * (2 * units + 24 + 48) * 2.0 ** -24, "dlogits")


@pytest.mark.gpu
def test_norm_calls_and_plain_form(ops):
    c = dict(T=7, H=448, dtype="bf16", residual=True)
    s, plain, got, exact = both(ops, dict(op="norm", codes=True, **c))
    y = exact["y"].cpu()
    for out in (plain, got):
        # the plain form adds 448 squares in any order: half of 448 steps through the root
        ref.assert_within(out["y"], y, ref.norm_y_bound(y, torch.bfloat16) + y.abs() * 2.0 ** -15,
                          "y")
        assert torch.equal(out["residual"], plain["residual"])
        want = (out["y"].float() / out["scale"][:, None]).to(torch.float8_e4m3fn)
        assert torch.equal(out["codes"].view(torch.uint8), want.view(torch.uint8))
    s, plain, got, exact = both(ops, dict(op="norm_backward", **c))
    h = [s[n].cpu() for n in ("dy", "dres", "h", "weight")]
    dx, dw, mx, mw = ref.norm_backward(*h, 1e-6)
    assert (exact["dx"].cpu() - dx).abs().max() <= 1e-12 * mx.max()
    for out in (plain, got):
        ref.assert_within(out["dx"], dx, ref.norm_dx_bound(dx, mx, torch.bfloat16)
                          + 2 * 448 * 2.0 ** -24 * mx, "dx")
        ref.assert_within(out["dweight"], dw, ref.norm_dw_bound(mw, 7) + 448 * 2.0 ** -24 * mw,
                          "dweight")
