"""The activation operators on matrices of more than 2^31 elements: offsets past 32 bits, checked on
rows from the start, around each 2^31st element and the end (and the weight gradient, a sum over all
rows, against exact sums)."""
import numpy as np
import pytest
import torch

import gradient_compression_amd as gca
import oracle
from tests.gpu_helpers import assert_bitwise, log

pytestmark = pytest.mark.gpu


def picked(rows, cols):
    """Rows around every 2^31 elements or bytes, the first and the last ones."""
    out = {0, 1, rows - 2, rows - 1}
    for e in (1 << 30, 1 << 31, 1 << 32):
        out |= {e // cols - 1, e // cols, e // cols + 1}
    return sorted(r for r in out if 0 <= r < rows)


def f32(t):
    return t.float().cpu().numpy()


def test_norm_and_checkpoint_of_a_long_matrix():
    rows, cols = 270_001, 8224          # 2.2e9 elements, an odd row count, a ragged last wave
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    for a in range(0, rows, 30_000):
        x[a:a + 30_000].normal_()
    pitch, groups = gca.act_layout(cols)
    codes = torch.empty(rows, pitch, dtype=torch.int8, device="cuda")
    exps = torch.empty(rows, groups, dtype=torch.uint8, device="cuda")
    rstd = torch.empty(rows, device="cuda")
    y = torch.empty_like(x)
    log("[act max] norm")
    gca.rmsnorm(x, y=y, rstd=rstd, codes=codes, exps=exps, stochastic=True, seed=4, step=9)
    torch.cuda.synchronize()
    at = picked(rows, cols)
    z = f32(x[at]) * rstd[at].cpu().numpy()[:, None]
    assert torch.equal(y[at].cpu(), torch.from_numpy(z).to(torch.bfloat16))
    # the draws go by the element's place in the whole matrix
    for r, row in zip(at, z):
        c = codes[r].cpu().numpy()
        _, e = oracle.act_quant(row[None])
        assert_bitwise(exps[r:r + 1], e, f"row {r} exponents")
        unit = np.ldexp(1.0, np.repeat(e[0].astype(int) - 127, 32))[:cols]
        a = np.abs(row.astype(np.float64)) / unit
        i = r * pitch + np.arange(cols)
        draw = np.array([oracle.philox4x32_10(
            np.array([b & 0xFFFFFFFF, b >> 32, 9, 0x54], np.uint32), np.array([4, 0], np.uint32))
            for b in range(int(i[0]) // 4, int(i[-1]) // 4 + 1)]).reshape(-1)[:cols] >> 8
        q = np.floor(a) + (draw < (a - np.floor(a)) * 2.0 ** 24)
        assert np.array_equal(c[:cols], np.where(row < 0, -q, q)), f"row {r} codes"
    del y
    log("[act max] write and read back")
    gca.act_quant(x, codes, exps)
    back = torch.empty_like(x)
    gca.act_restore(codes, exps, back)
    torch.cuda.synchronize()
    want_c, want_e = oracle.act_quant(f32(x[at]))
    assert_bitwise(codes[at], want_c, "codes")
    assert_bitwise(exps[at], want_e, "exponents")
    assert np.array_equal(f32(back[at]), oracle.act_restore(want_c, want_e, cols))
    log("[act max] norm backward")
    dx, dw = x, torch.empty(cols, device="cuda")
    one = torch.ones(rows, device="cuda")
    back.fill_(1.0)                      # dy
    gca.rmsnorm_backward(back, codes, exps, one, dx, dweight=dw)
    torch.cuda.synchronize()
    zz = oracle.act_restore(want_c, want_e, cols).astype(np.float64)
    want = 1.0 - zz * zz.mean(1, keepdims=True)
    # fp32 sums and products, then half a step of bf16
    assert (np.abs(f32(dx[at]) - want) <= 2.0 ** -8 * np.abs(want) * 1.01 + 1e-5 * np.abs(zz)).all()


def test_weight_grad_over_a_long_batch():
    rows, n_out, cols = 300_017, 7936, 96     # 2.4e9 elements of dy
    dy = torch.empty(rows, n_out, dtype=torch.bfloat16, device="cuda")
    for a in range(0, rows, 20_000):
        n = min(20_000, rows - a)
        dy[a:a + n] = torch.randint(-1, 2, (n, n_out), device="cuda", dtype=torch.int8)
    codes = torch.randint(-3, 4, (rows, cols), device="cuda", dtype=torch.int8)
    exps = torch.full((rows, cols // 32), 127, dtype=torch.uint8, device="cuda")
    dw = torch.empty(n_out, cols, device="cuda")
    log("[act max] weight gradient")
    gca.act_weight_grad(dy, codes, exps, dw)
    torch.cuda.synchronize()
    want = torch.zeros(n_out, cols, device="cuda", dtype=torch.float64)
    for a in range(0, rows, 20_000):          # whole numbers below 2^24: exact in fp32
        want += (dy[a:a + 20_000].float().t().contiguous() @ codes[a:a + 20_000].float()).double()
    assert torch.equal(dw.double(), want)


def whole(shape, most, dtype=torch.float32):
    return torch.randint(-most, most + 1, shape, device="cuda").to(dtype)


def test_weight_grad_of_far_apart_rows():
    """Rows of dy further apart than 2^24 elements, and a checkpoint row of more than 2^25 columns."""
    ld = (1 << 24) + 40
    buf = torch.zeros(5 * ld, dtype=torch.bfloat16, device="cuda")
    dy = buf.as_strided((5, 200), (ld, 1), 3)
    dy.copy_(whole((5, 200), 50))
    codes = torch.randint(-50, 51, (5, 96), device="cuda", dtype=torch.int8)
    exps = torch.full((5, 3), 127, dtype=torch.uint8, device="cuda")
    dw = torch.empty(200, 96, device="cuda")
    gca.act_weight_grad(dy, codes, exps, dw)
    assert torch.equal(dw, dy.float().t().contiguous() @ codes.float())
    cols = (1 << 25) + 70
    pitch, groups = gca.act_layout(cols)
    codes = torch.randint(-50, 51, (3, pitch), device="cuda", dtype=torch.int8)
    exps = torch.full((3, groups), 127, dtype=torch.uint8, device="cuda")
    dy = whole((3, 2), 50, torch.bfloat16)
    dw = torch.empty(2, cols, device="cuda")
    gca.act_weight_grad(dy, codes, exps, dw)
    want = sum(dy[m].float()[:, None] * codes[m, :cols].float() for m in range(3))
    assert torch.equal(dw, want)


def test_weight_grad_of_the_largest_matrix():
    n_out, cols, rows = 65536, 32767, 70         # 2^31 - 65536 weights
    dy = whole((rows, n_out), 20, torch.bfloat16)
    pitch, groups = gca.act_layout(cols)
    codes = torch.randint(-20, 21, (rows, pitch), device="cuda", dtype=torch.int8)
    exps = torch.full((rows, groups), 127, dtype=torch.uint8, device="cuda")
    dw = torch.empty(n_out, cols, device="cuda")
    log("[act max] largest weight matrix")
    gca.act_weight_grad(dy, codes, exps, dw)
    torch.cuda.synchronize()
    z = codes[:, :cols].float()
    for a in range(0, n_out, 8192):
        want = dy[:, a:a + 8192].float().t().contiguous() @ z
        assert torch.equal(dw[a:a + 8192], want), f"rows from {a}"
