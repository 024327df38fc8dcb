"""The E4M3 scale rule on the borders: s = 2^n, n the smallest integer with
448 * 2^n >= amax, 1 for amax = 0, n held to [-126, 120]."""
import math

import pytest
import torch

from sparse_moe_layer_06_b200 import moe

pytestmark = pytest.mark.gpu
DEV = "cuda"

NEXT = 1 + 2.0 ** -23
LARGEST = [0.0, 448.0, 448.0 * NEXT, 447.0, 1.75 * 2.0 ** -60, 1.75 * 2.0 ** -60 * NEXT, 1.0, 3.0,
           2.0 ** -126, 2.0 ** -118, 1.75 * 2.0 ** -118, 1.75 * 2.0 ** -118 * NEXT, 1e-40, 2.0 ** -149,
           torch.finfo(torch.float32).max, 1.75 * 2.0 ** 127, math.inf]


def scale(amax):
    if amax == 0:
        return 1.0
    if math.isinf(amax):
        return 2.0 ** 120
    n = -200
    while 448 * 2.0 ** n < amax:
        n += 1
    return 2.0 ** min(max(n, -126), 120)


def test_row_and_column_scales():
    H = I = 128
    p = moe.MoEProblem(T=1, H=H, E=1, I=I, top_k=1, num_shared=0, routed_scale=1.0,
                       clip_limit=10.0, dtype=torch.float32)
    w = torch.zeros(1, 3, I, H)
    part = torch.linspace(-1, 1, H)
    for i, a in enumerate(LARGEST):
        v = part * min(a, torch.finfo(torch.float32).max) * 0.5
        v[7] = a
        w[0, 0, i], w[0, 1, i], w[0, 2, :, i] = v, -v, v
    q = torch.empty(1, 3, I, H, dtype=torch.uint8, device=DEV)
    s_gu, s_d = torch.empty(1, 2, I, device=DEV), torch.empty(1, H, device=DEV)
    moe.moe_quantize_weights_fp8(p, w.to(DEV), q, s_gu, s_d)
    q, s_gu, s_d = q.cpu(), s_gu.cpu(), s_d.cpu()
    for i, a in enumerate(LARGEST):
        a = float(torch.tensor(a, dtype=torch.float32))
        assert s_gu[0, 0, i] == s_gu[0, 1, i] == s_d[0, i] == scale(a), a
        for m, got in ((w[0, 0, i], q[0, 0, i]), (w[0, 1, i], q[0, 1, i]),
                       (w[0, 2, :, i], q[0, 2, :, i])):
            # v / s is exact in 64 bits; torch has no saturation, so infinities are held to 448
            want = (m.double() / scale(a)).clamp(-448, 448).float().to(torch.float8_e4m3fn)
            assert torch.equal(got, want.view(torch.uint8)), a
