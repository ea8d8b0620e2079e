"""Pins of the oracle's 8-bit activation checkpoint: hand-worked groups, the properties of the
definition, the expectation of the stochastic rounding, and planted mistakes that the pins catch.
"""
import numpy as np
import pytest

import oracle

F = np.float32


def test_hand_worked_group():
    # A = 127 needs 2^0; one above it 2^1; ties go to even
    x = np.zeros((1, 64), F)
    x[0, :6] = [127.0, -0.5, 1.5, 2.5, -126.5, 0.49]
    x[0, 32:36] = [127.5, 1.0, 3.0, -5.0]
    codes, exps = oracle.act_quant(x)
    assert exps.tolist() == [[127, 128]]
    assert codes[0, :6].tolist() == [127, 0, 2, 2, -126, 0]
    assert codes[0, 32:36].tolist() == [64, 0, 2, -2]   # 63.75, 0.5, 1.5, -2.5
    assert not codes[0, 6:32].any() and not codes[0, 36:].any()
    assert oracle.act_restore(codes, exps, 64)[0, :3].tolist() == [127.0, 0.0, 2.0]
    assert oracle.act_restore(codes, exps, 64)[0, 32] == 128.0


def test_short_last_group_and_padding():
    x = np.arange(1, 36, dtype=F).reshape(1, 35)
    codes, exps = oracle.act_quant(x)
    assert codes.shape == (1, 64) and exps.shape == (1, 2)
    assert not codes[0, 35:].any()
    back = oracle.act_restore(codes, exps, 35)
    assert np.abs(back - x).max() <= 0.25   # 2^(e-1) with e = -1 (35 <= 127 / 2)


def test_ends_of_the_range():
    top = np.ldexp(F(127), 121).astype(F)
    x = np.zeros((6, 32), F)
    x[0, 3] = np.inf
    x[1, 0], x[1, 1] = np.nan, 5
    x[2, 7] = top
    x[3, 7] = np.nextafter(top, F(np.inf))
    x[4, 0], x[4, 1] = F(2.0 ** -120), F(2.0 ** -122)
    codes, exps = oracle.act_quant(x)
    assert exps[:, 0].tolist() == [255, 255, 248, 255, 7, 7]
    assert codes[2, 7] == 127 and codes[4, 0] == 1 and codes[4, 1] == 0
    for r in (0, 1, 3, 5):
        assert not codes[r].any()
    back = oracle.act_restore(codes, exps, 32)
    assert np.isnan(back[[0, 1, 3]]).all()
    assert back[2, 7] == top and not back[5].any()


@pytest.mark.parametrize("random", [False, True])
def test_error_within_a_step_and_codes_use_the_range(random):
    rng = np.random.default_rng(3)
    x = (rng.standard_t(3, (50, 100)) * np.exp(rng.normal(size=(50, 1)) * 8)).astype(F)
    codes, exps = oracle.act_quant(x, random=random, seed=5, step=9)
    assert np.abs(codes.astype(int)).max() <= 127
    back = oracle.act_restore(codes, exps, 100).astype(np.float64)
    unit = np.repeat(np.ldexp(1.0, exps.astype(int) - 127), 32, axis=1)[:, :100]
    assert (np.abs(back - x) <= (unit if random else unit / 2)).all()
    amax = np.abs(codes.reshape(50, -1, 32).astype(int)).max(2)
    assert (amax >= (63 if random else 64)).all()   # the smallest scale that holds the group
    if random:
        assert (np.abs(back - x) < unit).all()


def test_stochastic_rounding_is_unbiased_and_by_its_counter():
    x = np.full((4000, 32), 0.3, F)
    x[:, 0] = 127.0
    codes, exps = oracle.act_quant(x, random=True, seed=1, step=2)
    assert (exps == 127).all()
    got = codes[:, 1:].astype(float)
    assert set(np.unique(got)) == {0.0, 1.0}
    # 124000 draws of variance 0.21: five standard deviations
    assert abs(got.mean() - F(0.3)) < 5 * np.sqrt(0.21 / got.size)
    # element (m, c) takes word i % 4 of block i // 4, i = m * 32 + c
    for m, c in ((0, 1), (7, 30), (3999, 17)):
        i = m * 32 + c
        w = oracle.philox4x32_10(np.array([i // 4, 0, 2, 0x54], np.uint32),
                                 np.array([1, 0], np.uint32))[i % 4]
        assert codes[m, c] == int((int(w) >> 8) < float(F(0.3)) * 2 ** 24)
    other, _ = oracle.act_quant(x, random=True, seed=1, step=3)
    assert (other != codes).mean() > 0.3


MUTANTS = {
    "scale_one_too_large": ("while (!bad && most > ldexp(127.0, e)) ++e;",
                            "while (!bad && most > ldexp(63.0, e)) ++e;"),
    "scale_by_128": ("most > ldexp(127.0, e)", "most > ldexp(128.0, e)"),
    "ties_away": ("code = (int8_t)nearbyint(v);", "code = (int8_t)round(v);"),
    "draw_word_0": ("return r[i % 4] >> 8;", "return r[0] >> 8;"),
    "sign_lost": ("code = (int8_t)(v < 0.0 ? -q : q);", "code = (int8_t)q;"),
    "counter_without_pitch": ("act_draw24(seed, step, m * pitch + c)",
                              "act_draw24(seed, step, c)"),
    "nan_ignored": ("if (!isfinite(v)) bad = 1;", "if (isinf(v)) bad = 1;"),
}


@pytest.mark.parametrize("name", sorted(MUTANTS))
def test_planted_mistakes_are_caught(name, tmp_path, monkeypatch):
    old, new = MUTANTS[name]
    src = oracle.source()
    assert src.count(old) == 1
    so = oracle.compile_variant(src.replace(old, new), str(tmp_path / "mutant.so"))
    monkeypatch.setattr(oracle, "_lib", oracle.load(so))
    with pytest.raises(AssertionError):
        test_hand_worked_group()
        test_short_last_group_and_padding()
        test_ends_of_the_range()
        for random in (False, True):
            test_error_within_a_step_and_codes_use_the_range(random)
        test_stochastic_rounding_is_unbiased_and_by_its_counter()
