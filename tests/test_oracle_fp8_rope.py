"""The oracles of the block-scaled FP8 layer and of the rotary positions, against brute force, a second library
routine and invariants."""
import numpy as np
import pytest
import torch

from oracle import fp8, rope


def test_e4m3_codes_round_trip_and_match_torch():
    codes = np.array([c for c in range(256) if c & 127 != 127], dtype=np.uint8)
    v = fp8.decode(codes)
    assert np.array_equal(v, torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy())
    assert np.array_equal(fp8.encode(v), codes)
    grid = np.unique(v)
    # every midpoint, its neighbours, and a sweep: nearest by exhaustive search, ties to the even code
    mid = (grid[:-1] + grid[1:]) / 2
    u = np.concatenate([mid, np.nextafter(mid, 1e9), np.nextafter(mid, -1e9), np.linspace(-448, 448, 3001)])
    got = fp8.e4m3_round(u)
    d = np.abs(u[:, None] - grid)
    best = d.min(1)
    assert np.array_equal(np.abs(u - got), best)
    tie = (d == best[:, None]).sum(1) > 1
    assert (fp8.encode(got[tie]) % 2 == 0).all()


def test_scale_is_the_smallest_power_of_two():
    x = np.zeros((6, 128))
    x[0, 5], x[1, 7], x[2, 0], x[3, 1], x[4, 9] = 448.0, 449.0, 3.5, -3.5000001, 2.0 ** -133
    _, e = fp8.quantize(x)
    assert e[:, 0].tolist() == [0, 1, -7, -6, -127, -127]


def test_error_of_a_code_is_at_most_half_a_step():
    r = np.random.default_rng(0)
    x = r.normal(size=(50, 300)) * np.exp2(r.integers(-40, 40, size=(50, 1)).astype(float))
    q = fp8.value(x)
    _, e = fp8.quantize(x)
    s = np.repeat(np.exp2(e.astype(float)), 128, axis=1)[:, :300]
    assert (np.abs(q - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s)).all()


def test_non_finite_becomes_nan_and_leaves_the_block_scaled():
    x = np.ones((2, 256))
    x[0, 3], x[0, 4], x[1, 130] = np.inf, np.nan, -np.inf
    q = fp8.value(x)
    assert np.isnan(q[0, [3, 4]]).all() and np.isnan(q[1, 130]) and np.isnan(q).sum() == 3
    assert (q[~np.isnan(q)] == 1).all()


def test_linear_and_experts_by_loops():
    r = np.random.default_rng(1)
    x, w, b = r.normal(size=(7, 130)), r.normal(size=(3, 130, 4)), r.normal(size=(3, 4))
    off = [0, 2, 2, 6]
    y, mag = fp8.experts(x, w, off, b)
    for e in range(3):
        for m in range(off[e], off[e + 1]):
            for n in range(4):
                terms = [fp8.value(x[m:m + 1])[0, k] * fp8.value(w[e].T)[n, k] for k in range(130)]
                assert abs(sum(terms) + b[e, n] - y[m, n]) < 1e-12
                assert abs(sum(abs(t) for t in terms) + abs(b[e, n]) - mag[m, n]) < 1e-12
    assert np.isnan(y[6]).all()


@pytest.mark.parametrize("half", [False, True])
def test_rope_is_a_turn(half):
    r = np.random.default_rng(2)
    x, pos = r.normal(size=(5, 3, 16)), r.integers(0, 999, size=(5, 2))
    y = rope.rope(x, pos, [6, 10], half=half)
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
    assert np.allclose(rope.rope(y, pos, [6, 10], half=half, inverse=True), x)
    # products of two turned heads depend on the difference of their positions alone
    z = rope.rope(x, pos + 17, [6, 10], half=half)
    y0, z0 = rope.rope(x[:, :1], pos, [6, 10], half=half), rope.rope(x[:, 1:2], pos, [6, 10], half=half)
    y1, z1 = rope.rope(x[:, :1], pos + 17, [6, 10], half=half), rope.rope(x[:, 1:2], pos + 17, [6, 10], half=half)
    assert np.allclose((y0 * z0).sum(-1), (y1 * z1).sum(-1)) and not np.allclose(y, z)
    # by hand: the second axis' first pair is pair 3, frequency 1
    i, j = (3, 11) if half else (6, 7)
    p = pos[2, 1]
    assert np.isclose(y[2, 1, i], x[2, 1, i] * np.cos(p) - x[2, 1, j] * np.sin(p))
    assert np.isclose(y[2, 1, j], x[2, 1, i] * np.sin(p) + x[2, 1, j] * np.cos(p))
