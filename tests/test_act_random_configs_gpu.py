"""The activation operators over seeded random sizes, types, strides and options, each call compared
as in tests/test_act_gpu.py (whose checks derive the tolerances)."""
import random

import pytest
import torch

from tests.gpu_helpers import log
from tests import test_act_gpu as T

pytestmark = pytest.mark.gpu


def size(rng, low, high):
    return int(round(low * (high / low) ** rng.random()))


@pytest.mark.parametrize("seed", range(12))
def test_norm_and_checkpoint(seed):
    rng = random.Random(seed)
    for i in range(8):
        rows, cols = size(rng, 1, 2000), size(rng, 1, 12000)
        rows = max(1, min(rows, 2_000_000 // cols))
        dtype = rng.choice(sorted(T.TYPES))
        label = f"{seed}.{i} {dtype} {rows}x{cols}"
        log(f"[random] {label}")
        x = T.activations(rows, cols, dtype, 100 * seed + i)
        if rng.random() < 0.5:
            x, _ = T.strided(x, rng.randrange(0, 40), rng.randrange(0, 8))
        res = T.activations(rows, cols, dtype, 7 * i) if rng.random() < 0.5 else None
        w = (torch.rand(cols, device="cuda") + 0.5).to(T.TYPES[rng.choice(sorted(T.TYPES))])
        h, y = torch.empty_like(x), torch.empty(rows, cols, dtype=x.dtype, device="cuda")
        T.check_norm(x, res, w if rng.random() < 0.8 else None, rng.choice([1e-6, 1e-3]), dtype,
                     h=h if res is not None else None, y=y, random=rng.random() < 0.4, label=label)
        T.check_quant(x, rng.random() < 0.4, label)
        T.check_backward(rows, cols, dtype, seed + i, residual=rng.random() < 0.6,
                         weight=rng.choice([None, "f32", "bf16", "f16"]),
                         accumulate=rng.random() < 0.5, pad=rng.choice([None, 0, 1, 5, 8]))


@pytest.mark.parametrize("seed", range(12))
def test_weight_grad(seed):
    rng = random.Random(1000 + seed)
    for i in range(6):
        rows, n_out, cols = size(rng, 1, 5000), size(rng, 1, 3500), size(rng, 1, 3500)
        rows = max(1, min(rows, 3_000_000_000 // (n_out * cols)))
        dtype = rng.choice(sorted(T.TYPES))
        log(f"[random] {seed}.{i} {dtype} {rows} {n_out}x{cols}")
        dy, codes, exps, want = T.exact_case(rows, n_out, cols, dtype, seed + i)
        if rng.random() < 0.5:
            dy, _ = T.strided(dy, rng.randrange(0, 40), rng.randrange(0, 8))
        flat = torch.full((n_out * cols + 2,), 7.0, device="cuda")
        at = rng.randrange(0, 3)
        dw = flat[at:at + n_out * cols].view(n_out, cols)
        dw.fill_(1.0)
        add = rng.random() < 0.5
        T.gca.act_weight_grad(dy, codes, exps, dw, accumulate=add)
        torch.cuda.synchronize()
        assert T.np.array_equal(T.f64(dw), want + (1.0 if add else 0.0))
        assert bool((flat[:at] == 7.0).all()) and bool((flat[at + n_out * cols:] == 7.0).all())
