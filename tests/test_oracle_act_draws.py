"""What stochastic checkpoints share: the draws are those of (seed, step, place in the matrix), so
matrices written with the same seed and step are rounded alike, and others independently."""
import numpy as np

import oracle


def errors(x, seed, step):
    """What the rounding adds to each magnitude, in units of its scale: [u < f] - f with f the
    magnitude's fraction."""
    codes, exps = oracle.act_quant(x, random=True, seed=seed, step=step)
    unit = np.repeat(np.ldexp(1.0, exps.astype(int) - 127), 32, axis=1)[:, :x.shape[1]]
    back = oracle.act_restore(codes, exps, x.shape[1]).astype(np.float64)
    return (back - x) * np.sign(x) / unit


def test_draws_go_by_seed_step_and_place():
    rng = np.random.default_rng(1)
    a, b = (rng.normal(size=(200, 96)).astype(np.float32) for _ in range(2))
    same = np.corrcoef(errors(a, 7, 3).ravel(), errors(b, 7, 3).ravel())[0, 1]
    # errors of independent roundings: a correlation's deviation is 1 / sqrt(19200) = 0.0072; with
    # shared draws u, errors [u < f] - f of uniform fractions f, g: covariance 1/12 of variance 1/6
    assert abs(same - 0.5) < 6 * 0.0072
    for seed, step in ((8, 3), (7, 4), (7 + (1 << 32), 3)):
        other = np.corrcoef(errors(a, 7, 3).ravel(), errors(b, seed, step).ravel())[0, 1]
        assert abs(other) < 6 * 0.0072
    # only the step's low 32 bits count
    assert np.array_equal(errors(a, 7, 3), errors(a, 7, 3 + (1 << 32)))


def test_errors_of_micro_batches_average_out_with_their_own_steps():
    x = np.random.default_rng(2).normal(size=(64, 64)).astype(np.float32)
    one = np.sqrt(np.mean(errors(x, 7, 0) ** 2))
    own = np.sqrt(np.mean(np.mean([errors(x, 7, t) for t in range(16)], 0) ** 2))
    shared = np.sqrt(np.mean(np.mean([errors(x, 7, 0) for _ in range(16)], 0) ** 2))
    assert shared == one
    # the mean of 16 independent errors: a quarter; 4096 values, each side within 10 %
    assert abs(own / one - 0.25) < 0.025
