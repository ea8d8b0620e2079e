"""The norm's backward pass where every worker takes several rows: its sums over rows, the row loaded
ahead, the two places of the waves' sums (an even and an odd number of rows), and the non-temporal
loads of large gradients, each with a weight, the residual's gradient and an accumulated weight
gradient, against the formula in 64 bits on the device."""
import pytest
import torch

import gradient_compression_amd as gca
from tests.gpu_helpers import log

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}      # half a step, relative
SMALLEST = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}
U = 2.0 ** -24


def checkpoint(gen, rows, cols):
    """Random codes and scales, zeros behind the last column; and their values in 64 bits."""
    pitch, groups = gca.act_layout(cols)
    codes = torch.randint(-127, 128, (rows, pitch), generator=gen, device="cuda", dtype=torch.int8)
    codes[:, cols:] = 0
    exps = torch.randint(119, 123, (rows, groups), generator=gen, device="cuda", dtype=torch.uint8)
    return codes, exps


def values(codes, exps, cols):
    unit = ((exps.long() + (1023 - 127)) << 52).view(torch.float64)      # 2^(exps - 127)
    return (codes.double().view(*exps.shape, 32) * unit[:, :, None]).flatten(1)[:, :cols]


def check(rows, cols, dtype, weight, residual, accumulate, pad, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    codes, exps = checkpoint(gen, rows, cols)
    matrix = lambda: (normal(rows, cols + pad) * 1e-2).to(TYPES[dtype])[:, :cols]  # noqa: E731
    dy, dres = matrix(), matrix() if residual else None
    w = (1.0 + 0.2 * normal(cols)).to(TYPES[weight]) if weight else None
    rstd = torch.rand(rows, generator=gen, device="cuda") + 0.5
    start = normal(cols)
    dw = start.clone()
    wide = torch.full((rows, cols + pad), 7.0, dtype=TYPES[dtype], device="cuda")
    dx = wide[:, :cols]
    gca.rmsnorm_backward(dy, codes, exps, rstd, dx, weight=w, dres=dres, dweight=dw,
                         accumulate=accumulate)
    torch.cuda.synchronize()
    assert bool((wide[:, cols:] == 7.0).all())
    total = torch.zeros(cols, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(total)
    hw = 1.0 if w is None else w.double()
    step = max(1, (1 << 25) // cols)
    for a in range(0, rows, step):
        z, g = values(codes[a:a + step], exps[a:a + step], cols), dy[a:a + step].double()
        r = rstd[a:a + step].double()[:, None]
        t = g * hw
        c = (t * z).mean(1, keepdim=True)
        want = r * (t - z * c)
        if residual:
            want += dres[a:a + step].double()
        # t one rounding, the sum 32 terms deep in a lane, 6 in its wave, 16 over the waves, the
        # quotient one; then the difference, the product and the sum one each; 1 % for second orders
        c_err = 1.01 * (32 + 6 + 16 + 2) * U * (t * z).abs().mean(1, keepdim=True)
        tol = (1.01 * (r * (3 * U * (t.abs() + (z * c).abs()) + z.abs() * c_err)
                       + 2 * U * want.abs() + HALF[dtype] * want.abs()) + SMALLEST[dtype] / 2)
        if residual:
            tol += 1.01 * U * dres[a:a + step].double().abs()
        off = (dx[a:a + step].double() - want).abs()
        assert bool((off <= tol).all()), f"dx off by {float((off / tol).max())} of its tolerance"
        total += (g * z).sum(0)
        size += (g * z).abs().sum(0)
    # a worker's rows one after the other (256 blocks or more, or one row each), the four waves of a
    # block, up to 1024 blocks in 128 slices, three steps in a wave, 16 waves, the accumulation
    deep = -(-rows // 256) + 3 + 8 + 3 + 16 + 1
    want = total + (start.double() if accumulate else 0.0)
    tol = 1.01 * U * (deep * size + (start.double().abs() if accumulate else 0.0) + want.abs())
    off = (dw.double() - want).abs()
    assert bool((off <= tol).all()), f"dw off by {float((off / tol).max())} of its tolerance"
    return dx, dw


# one case for each width of workers; some workers of a case take one row more than the others, three
# or four in all
WIDTHS = [(3077, 500), (3079, 1001), (3076, 2000), (770, 4095), (773, 8192), (771, 12000), (769, 16383),
          (774, 32768)]


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("rows,cols", WIDTHS)
def test_workers_of_several_rows(rows, cols, dtype):
    log(f"[norm rows] {dtype} {rows}x{cols}")
    check(rows, cols, dtype, weight=dtype, residual=True, accumulate=True, pad=0, seed=1)
    check(rows, cols, dtype, weight=None, residual=False, accumulate=False, pad=0, seed=2)
    check(rows, cols, dtype, weight="f32", residual=True, accumulate=False, pad=5, seed=3)


# at least 32 MB of gradients in every type
LARGE = [(33001, 509), (17001, 1000), (8501, 2048), (4101, 4096), (2101, 8184), (1501, 12000),
         (1100, 16384), (520, 32767)]


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("rows,cols", LARGE)
def test_large_gradients(rows, cols, dtype):
    log(f"[norm rows] {dtype} {rows}x{cols}")
    assert rows * cols * 2 >= 32 << 20
    check(rows, cols, dtype, weight="bf16", residual=True, accumulate=True, pad=0, seed=4)
    check(rows, cols, dtype, weight=dtype, residual=False, accumulate=True, pad=3, seed=5)


def test_more_than_2_to_31_elements():
    log("[norm rows] 270001x8224")
    check(270_001, 8224, "bf16", weight="f32", residual=True, accumulate=True, pad=0, seed=6)
