"""Rotary positions over several axes on the GPU, against the float64 oracle.

Tolerance: cos and sin are float64 values rounded to fp32 (2^-24 each), each output is two products and one sum in
fp32, so 4 * 2^-24 of |x| + |y| for a pair (x, y); with a norm, x carries the norm's own error: a sum of D squares in
fp32 (D 2^-24 relative, halved by the root), the reciprocal root (2^-22) and three products.  Then bf16's half step."""
import numpy as np
import pytest
import torch

from bit_w4a4_diffusion_smooth_b200 import layer, lib
from oracle import rope
from tests import gpu_util as G

pytestmark = pytest.mark.gpu
AXES = {8: [8], 24: [8, 16], 64: [16, 24, 24], 80: [80], 128: [44, 42, 42], 256: [64, 96, 96], 136: [8, 128]}


@pytest.fixture(scope="module", autouse=True)
def _init():
    G.init()


def rand(seed, *shape):
    return torch.from_numpy(np.random.default_rng(seed).normal(size=shape).astype(np.float32)).to(torch.bfloat16).to(G.DEV)


def f64(t):
    return t.double().cpu().numpy()


def close(got, x, pos, axes, half, inverse=False, w=None, eps=1e-6, theta=10000.0):
    x = f64(x)
    want = rope.rope(x, f64(pos), axes, theta, half, inverse, None if w is None else f64(w), eps)
    v = np.abs(x if w is None else rope.norm(x, f64(w), eps))
    n = v.shape[-1] // 2
    a, b = (v[..., :n], v[..., n:]) if half else (v[..., 0::2], v[..., 1::2])
    s = a + b
    pair = np.concatenate([s, s], -1) if half else np.repeat(s, 2, -1)
    rel = 4 * 2.0 ** -24 + (0 if w is None else (x.shape[-1] / 2 + 8) * 2.0 ** -24)
    tol = rel * pair + 2.0 ** -8 * (np.abs(want) + rel * pair) + 2.0 ** -134
    bad = ~(np.abs(f64(got) - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), f64(got)[bad][:4], want[bad][:4])


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("D", sorted(AXES))
@pytest.mark.parametrize("M,hq,hk", [(1, 1, 1), (5, 8, 2), (701, 3, 1), (66, 20, 20)])
def test_against_oracle(half, normed, D, M, hq, hk):
    axes = AXES[D]
    qkv = rand(D + M, M, (hq + 2 * hk) * D)                    # heads of a fused projection: strided views
    q, k = qkv[:, :hq * D].unflatten(1, (hq, D)), qkv[:, hq * D:(hq + hk) * D].unflatten(1, (hk, D))
    w = [rand(i, D) for i in (1, 2)] if normed else [None, None]
    turn = layer.RotaryND(axes, interleaved=not half, q_norm=w[0], k_norm=w[1])
    pos = torch.randint(0, 5000, (M, len(axes)), device=G.DEV, dtype=torch.int32)
    qo, ko = turn(q, k, pos)
    G.check_ok()
    close(qo, q, pos, axes, half, w=w[0])
    close(ko, k, pos, axes, half, w=w[1])
    if not normed:
        qi, ki = turn(q, k, pos, inverse=True)
        close(qi, q, pos, axes, half, inverse=True)
        close(ki, k, pos, axes, half, inverse=True)


def test_far_and_fractional_positions():
    """Angles where a float32 product would be off by whole turns; positions between the whole ones."""
    axes = [64, 64]
    x = rand(1, 40, 2, 128)
    turn = layer.RotaryND(axes)
    far = torch.randint(-2 ** 31, 2 ** 31 - 1, (40, 2), device=G.DEV, dtype=torch.int64).to(torch.int32)
    close(turn(x, None, far)[0], x, far, axes, False)
    frac = torch.rand(40, 2, device=G.DEV) * 1e6
    close(turn(x, None, frac)[0], x, frac, axes, False)
    slow = layer.RotaryND(axes, theta=1e7, interleaved=False)
    close(slow(x, None, frac)[0], x, frac, axes, True, theta=1e7)


def test_one_normed_side():
    x, w = rand(1, 30, 3, 64), rand(2, 64)
    pos = torch.arange(30, device=G.DEV, dtype=torch.int32)[:, None].expand(30, 2)
    assert pos.stride(1) == 0
    with pytest.raises(ValueError):
        layer.RotaryND([32, 32])(x, x, pos)                   # axes that share memory are not unit-strided
    pos = pos.contiguous()
    turn = layer.RotaryND([32, 32], q_norm=w)
    q, k = turn(x, x, pos)
    close(q, x, pos, [32, 32], False, w=w)
    close(k, x, pos, [32, 32], False)
    with pytest.raises(lib.SvdqError):
        turn(x, x, pos, inverse=True)


@pytest.mark.parametrize("half", [False, True])
def test_in_place_layouts_and_untouched_bytes(half):
    M, H, D = 90, 3, 64
    turn = layer.RotaryND([16, 24, 24], interleaved=not half)
    pos = torch.randint(0, 99, (M, 5), device=G.DEV, dtype=torch.int32)[:, 1:4]      # strided rows
    qkv = rand(1, M, 3 * H * D)
    q, k = (qkv[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in range(2))
    want_q, want_k = turn(q, k, pos)
    close(want_q, q, pos, [16, 24, 24], half)
    # into [heads, rows, D], the layout of a batched attention
    hq = G.poisoned_bf16(H, M + 1, D)
    turn(q, k, pos, q_out=hq[:, :M].transpose(0, 1), k_out=torch.empty_like(want_k))
    assert torch.equal(hq[:, :M].transpose(0, 1), want_q) and torch.isnan(hq[:, M]).all()
    # in place: the value heads stay
    v = qkv[:, 2 * H * D:].clone()
    q2, k2 = turn(q, k, pos, q_out=q, k_out=k)
    assert q2 is q and torch.equal(q, want_q) and torch.equal(k, want_k) and torch.equal(qkv[:, 2 * H * D:], v)
    G.check_ok()


@pytest.mark.parametrize("half", [False, True])
def test_inverse_undoes_and_is_the_gradient(half):
    """<turn(x), g> = <x, turn_back(g)> is what makes the inverse the turn's gradient: held in the oracle to 1e-12
    and against differences, and on the GPU against the oracle's gradient."""
    r = np.random.default_rng(0)
    axes, M, H, D = [16, 24, 24], 20, 2, 64
    x, g, pos = r.normal(size=(M, H, D)), r.normal(size=(M, H, D)), r.integers(0, 500, size=(M, 3))
    grad = rope.rope(g, pos, axes, half=half, inverse=True)
    loss = lambda x: (rope.rope(x, pos, axes, half=half) * g).sum()
    assert abs((grad * x).sum() - loss(x)) < 1e-9
    for i in r.integers(0, x.size, size=20):
        d = np.zeros(x.size)
        d[i] = 1e-3
        d = d.reshape(x.shape)
        assert abs((loss(x + d) - loss(x - d)) / 2e-3 - grad.reshape(-1)[i]) < 1e-8
    G_ = torch.from_numpy(g).to(torch.bfloat16).to(G.DEV)
    P = torch.from_numpy(pos).to(torch.int32).to(G.DEV)
    back = layer.RotaryND(axes, interleaved=not half)(G_, None, P, inverse=True)[0]
    close(back, G_, P, axes, half, inverse=True)


def test_non_finite_stays_in_its_head():
    turn, normed = layer.RotaryND([64]), layer.RotaryND([64], q_norm=rand(3, 64))
    x = rand(1, 10, 3, 64)
    pos = torch.arange(10, device=G.DEV, dtype=torch.int32)[:, None]
    x[4, 1, 10], x[7, 2, 33] = float("nan"), float("inf")
    nan = torch.isnan(turn(x, None, pos)[0]) | torch.isinf(turn(x, None, pos)[0])
    want = torch.zeros_like(nan)
    want[4, 1, 10:12] = True
    want[7, 2, 32:34] = True
    assert torch.equal(nan, want)
    bad = torch.isnan(normed(x, None, pos)[0]).any(-1)
    want = torch.zeros_like(bad)
    want[4, 1] = want[7, 2] = True
    assert torch.equal(bad, want)


def test_refusals():
    turn = layer.RotaryND([32, 32])
    x, pos = rand(1, 6, 2, 64), torch.zeros(6, 2, dtype=torch.int32, device=G.DEV)
    for call in (lambda: turn(x[..., :32], None, pos), lambda: turn(x, None, pos[:, :1]), lambda: turn(x, None, pos[:5]),
                 lambda: turn(x, x[:5], pos), lambda: turn(x.float(), None, pos), lambda: turn(x, None, pos.long()),
                 lambda: turn(x.cpu(), None, pos), lambda: turn(x, None, pos.cpu()), lambda: turn(x[0], None, pos),
                 lambda: turn(x, None, pos, k_out=x), lambda: turn(x, None, pos, q_out=x[:, :1]),
                 lambda: turn(x.transpose(1, 2).contiguous().transpose(1, 2), None, pos),
                 lambda: layer.RotaryND([32, 32], q_norm=rand(1, 32))):
        with pytest.raises(ValueError):
            call()
    odd = torch.zeros(6 * 2 * 64 + 4, dtype=torch.bfloat16, device=G.DEV)[4:].view(6, 2, 64)
    for call in (lambda: turn(odd, None, pos), lambda: turn(x, None, pos, q_out=x[:1].expand(6, 2, 64)),
                 lambda: turn(x[:0], None, pos[:0])):
        with pytest.raises(lib.SvdqError):
            call()


def test_outputs_on_top_of_other_inputs_and_misaligned_norms():
    turn = layer.RotaryND([32, 32])
    q, k, pos = rand(1, 6, 2, 64), rand(2, 6, 2, 64), torch.zeros(6, 2, dtype=torch.int32, device=G.DEV)
    for kw in (dict(q_out=k, k_out=q), dict(q_out=k), dict(k_out=q), dict(q_out=q, k_out=q)):
        with pytest.raises(lib.SvdqError):
            turn(q, k, pos, **kw)
    w = rand(3, 64)
    off = torch.zeros(67, dtype=torch.bfloat16, device=G.DEV)
    off[3:] = w
    a, b = layer.RotaryND([32, 32], q_norm=off[3:], k_norm=off[3:]), layer.RotaryND([32, 32], q_norm=w, k_norm=w)
    for x, y in zip(a(q, k, pos), b(q, k, pos)):
        assert torch.equal(x, y)
    G.check_ok()


def test_streams_and_graphs():
    turn = layer.RotaryND([44, 42, 42])
    x = rand(1, 800, 4, 128)
    pos = torch.randint(0, 900, (800, 3), device=G.DEV, dtype=torch.int32)
    want = turn(x, x, pos)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = turn(x, x, pos, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = turn(x, x, pos)
    pos.add_(3)
    g.replay()
    torch.cuda.synchronize()
    close(out[0], x, pos, [44, 42, 42], False)
    G.check_ok()


def test_rows_past_32_bit_offsets():
    M, H, D = 70000, 128, 128                                  # 2.3 GB a tensor
    base = rand(1, 16, H, D)
    x = base.repeat(M // 16, 1, 1)
    pos = torch.arange(M, device=G.DEV, dtype=torch.int32)[:, None]
    out = layer.RotaryND([128])(x, None, pos)[0]
    rows = torch.tensor([0, 16, 65535, 65536, 65537, M - 1], device=G.DEV)
    assert M * H * D * 2 > 2 ** 31
    close(out[rows], x[rows], pos[rows], [128], False)


# Error of the kernel's turn, before bf16: the angle's product with the frequency and its remainder within half a turn are
# float64 with their rounding errors carried (2^-50 of a radian for any position), its float32 remainder's own error (up to
# 2^-26 turns) goes back into cosine and sine as a first-order term (what that leaves out: below 2^-46), sincospif is off by
# one unit in the last place at most (2^-23 of the value), and that correction, the product and the sum round once each
# (2^-24).  Of x cos - y sin that is 6 * 2^-24 of |x cos| + |y sin| <= |x| + |y|, plus 2^-45 of it.

def extended(x, pos, turn, half, inverse=False):
    """(x, y) turned in 80-bit arithmetic by the frequencies of the layer's plan; and |x cos| + |y sin|."""
    x, pos = f64(x), f64(pos).astype(np.longdouble)
    n = x.shape[-1] // 2
    freq = np.array(turn.plan.freq[:n], dtype=np.longdouble)
    angle = (pos[:, np.array(turn.plan.axis[:n], dtype=np.int64)] * freq)[:, None, :] * (-1 if inverse else 1)
    c, s = np.cos(angle), np.sin(angle)
    a, b = (x[..., :n], x[..., n:]) if half else (x[..., 0::2], x[..., 1::2])
    join = lambda u, v: np.concatenate([u, v], -1) if half else np.stack([u, v], -1).reshape(x.shape)
    return join(a * c - b * s, a * s + b * c), join(abs(a * c) + abs(b * s), abs(a * s) + abs(b * c))


def close_extended(got, x, pos, turn, half, inverse=False):
    want, mag = extended(x, pos, turn, half, inverse)
    d = 6 * 2.0 ** -24 * mag + 2.0 ** -45 * (1 + mag)
    bad = ~(np.abs(f64(got) - want) <= d + 2.0 ** -8 * (np.abs(want) + d) + 2.0 ** -134)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), f64(got)[bad][:4], want[bad][:4])


@pytest.mark.parametrize("half", [False, True])
def test_angles_next_to_a_quarter_turn(half):
    """Where a cosine or a sine is small its value is the angle's distance from the quarter turns: float32 positions next
    to odd and even multiples of pi / 2, and whole ones that come near them, turning (1, 0)."""
    k = torch.arange(1, 700, dtype=torch.float64)
    near = (k * (np.pi / 2)).float()
    pos = torch.cat([near, torch.nextafter(near, torch.tensor(0.0)), -near,
                     torch.tensor([11., 22., 355., 710., 52174., 103993., 104348., 208341., 5419351.])])[:, None].to(G.DEV)
    x = torch.zeros(pos.shape[0], 1, 8, dtype=torch.bfloat16, device=G.DEV)
    x[..., 0] = 1
    turn = layer.RotaryND([8], interleaved=not half)
    for inverse in (False, True):
        got = turn(x, None, pos, inverse=inverse)[0]
        G.check_ok()
        close_extended(got, x, pos, turn, half, inverse)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("kind", ["int", "fraction", "large float"])
def test_far_positions_keep_their_angles(half, kind):
    r = np.random.default_rng(5)
    axes, M = [32, 64, 32], 300
    pos = {"int": r.integers(-2 ** 31, 2 ** 31, size=(M, 3)).astype(np.int32),
           "fraction": (r.random((M, 3)) * 2e6 - 1e6).astype(np.float32),
           "large float": (r.normal(size=(M, 3)) * 2.0 ** 40).astype(np.float32)}[kind]
    if kind == "int":
        pos[0], pos[1], pos[2] = -2 ** 31, 2 ** 31 - 1, 0
    pos, x = torch.from_numpy(pos).to(G.DEV), rand(6, M, 2, 128)
    turn = layer.RotaryND(axes, interleaved=not half)
    got = turn(x, None, pos)[0]
    G.check_ok()
    if kind == "large float":           # the 80-bit product of 2^42 is itself off by 2^-22
        want, mag = extended(x, pos, turn, half)
        assert (np.abs(f64(got) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * (1 + mag)).all()
    else:
        close_extended(got, x, pos, turn, half)
