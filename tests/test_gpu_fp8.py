"""Block-scaled FP8 on the GPU: the quantizer bit for bit, the linear layer and the product by expert against the
float64 oracle.

Tolerance of an output, before its bf16 rounding: every one of the K products and the bias enters one fp32 sum,
whose adds are off by at most one unit in the last place each (2^-23 of the largest partial sum, itself at most
S = sum |terms|), so (K + 2) 2^-23 S; the GELUs have slopes below 1.13 and their approximations are off by less
than 2e-6 (1 + |y|).  The rounding to bf16 adds half a step, 2^-8 of the value (2^-134 for the smallest)."""
import numpy as np
import pytest
import torch

from bit_w4a4_diffusion_smooth_b200 import layer, lib
from oracle import fp8, rope
from tests import gpu_util as G

pytestmark = pytest.mark.gpu
EPI = [lib.EPILOGUE_NONE, lib.EPILOGUE_GELU_ERF, lib.EPILOGUE_GELU_TANH]


@pytest.fixture(scope="module", autouse=True)
def _init():
    G.init()


def bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16)


def rand(seed, *shape, scale=1.0, loud=True):
    """bf16 values (as float64) with one in fifty columns twenty times as large."""
    r = np.random.default_rng(seed)
    x = r.normal(size=shape) * scale
    if loud:
        x = np.where(r.random(shape[-1]) < 0.02, 20 * x, x)
    return bf16(x).double().numpy()


def close(got, want, mag, K, epilogue):
    got = G.bf16_host(got)
    d = (K + 2) * 2.0 ** -23 * mag * 1.13
    if epilogue:
        d = d + 2e-6 * (1 + np.abs(want))
    tol = d + 2.0 ** -8 * (np.abs(want) + d) + 2.0 ** -134
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("M,K,ldx", [(1, 8, 8), (3, 136, 136), (9, 512, 520), (37, 640, 648), (64, 264, 264),
                                     (130, 1032, 1032), (128, 1032, 1040), (2, 4104, 4112), (3000, 264, 264)])
def test_quantizer_bit_for_bit(M, K, ldx):
    """Against the identity the layer returns q(X) itself: a code's 4 bits fit bf16, and the identity's codes are
    exact."""
    x = rand(M + K, M, K) * np.exp2(np.random.default_rng(1).integers(-20, 20, size=(M, 1)).astype(float))
    x[0, :min(K, 128)] = 0
    if M > 2:
        x[1, 0], x[1, 1] = 2.0 ** -110, -2.0 ** -112            # a block far below the others
        x[2, 0], x[2, 1], x[2, -1] = 3e38, -1e30, 448
    if M > 8:
        x[8, 0], x[8, 1] = 448, 0.875                           # a maximum that is just 448 * 2^0
    t = torch.full((M, ldx), 7.0, dtype=torch.bfloat16)
    t[:, :K] = bf16(x)
    Y = layer.FP8Linear(torch.eye(K, dtype=torch.bfloat16, device=G.DEV))(t.to(G.DEV)[:, :K])
    G.check_ok()
    want = fp8.value(bf16(x).double().numpy())
    assert np.array_equal(G.bf16_host(Y), want)


def test_smallest_magnitudes():
    """Subnormal inputs under the smallest scale: the code's value, or zero where the tensor core flushes a
    subnormal sum."""
    x = np.zeros((4, 128))
    x[0, 0], x[1, 1], x[2, 2], x[3, 3] = 2.0 ** -133, 3 * 2.0 ** -130, -2.0 ** -127, 2.0 ** -126
    Y = G.bf16_host(layer.FP8Linear(torch.eye(128, dtype=torch.bfloat16, device=G.DEV))(bf16(x).to(G.DEV)))
    want = fp8.value(x)
    assert ((Y == want) | ((Y == 0) & (np.abs(want) < 2.0 ** -126))).all() and Y[3, 3] == 2.0 ** -126


def run_linear(x, w, b, epilogue=0, begin=0, ldx=None, ldy=None):
    M, K = x.shape
    N = w.shape[1]
    X = torch.full((M, ldx or K), 7.0, dtype=torch.bfloat16)
    X[:, :K] = bf16(x)
    lin = layer.FP8Linear(bf16(w).to(G.DEV), None if b is None else bf16(b).to(G.DEV), epilogue, begin)
    Yf = G.poisoned_bf16(M, ldy or N)
    Y = lin(X.to(G.DEV)[:, :K], Yf[:, :N])
    G.check_ok()
    return Y, Yf


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 32, 33, 64, 65, 127, 128, 129, 300])
@pytest.mark.parametrize("K,N,epilogue", [(136, 264, 0), (520, 136, 1), (1416, 8, 2)])
def test_linear(M, K, N, epilogue):
    x, w, b = rand(M, M, K), rand(K, K, N, scale=0.05, loud=False), rand(N, N, loud=False)
    Y, _ = run_linear(x, w, b, epilogue)
    want, mag = fp8.linear(x, w, b, epilogue)
    close(Y, want, mag, K, epilogue)


@pytest.mark.parametrize("M,K,N", [(1, 8, 8), (5, 128, 128), (20, 8, 4104), (100, 2560, 512), (700, 4096, 264),
                                   (1000, 72, 1032), (257, 1024, 512), (513, 640, 768),
                                   # wide enough for the SM pairs' 256 x 240 tiles: one stage, a short last set of
                                   # scale words, several tiles a pair, ragged rows and columns
                                   (4000, 128, 9608), (2600, 1416, 5640), (5001, 640, 7688), (9000, 264, 3608)])
def test_linear_shapes(M, K, N):
    x, w = rand(M + 1, M, K), rand(K + 1, K, N, scale=0.05, loud=False)
    Y, _ = run_linear(x, w, None)
    close(Y, *fp8.linear(x, w), K, 0)


@pytest.mark.parametrize("M,N", [(3, 392), (40, 392), (200, 392), (600, 392), (3001, 7688)])
def test_linear_strides_gelu_begin_and_untouched_bytes(M, N):
    K = 264
    x, w, b = rand(5, M, K), rand(6, K, N, scale=0.05, loud=False), rand(7, N, loud=False)
    Y, Yf = run_linear(x, w, b, 1, 130, ldx=K + 24, ldy=N + 40)
    want, mag = fp8.linear(x, w, b, 1, 130)
    close(Y, want, mag, K, 1)
    assert torch.isnan(Yf[:, N:]).all()


@pytest.mark.parametrize("M,N", [(1, 400), (24, 400), (130, 400), (1030, 400), (2500, 8000)])
def test_linear_exact_on_small_integers(M, N):
    """Integers up to 8 are e4m3 values under any scale that keeps them normal; their sums fit 24 bits, so the
    result is the exact sum's bf16."""
    r = np.random.default_rng(M)
    K = 1304
    x, w = r.integers(-8, 9, size=(M, K)).astype(float), r.integers(-8, 9, size=(K, N)).astype(float)
    Y, _ = run_linear(x, w, None)
    assert torch.equal(Y.cpu(), bf16(x @ w))


@pytest.mark.parametrize("M,N", [(4, 264), (150, 264), (1100, 264), (4000, 6008)])
def test_scales_of_every_block_and_row(M, N):
    """Each row and each block of 128 at a magnitude of its own: a scale taken for another row or block shows."""
    r = np.random.default_rng(3)
    K = 1160
    KS = -(-K // 128)
    x = r.integers(1, 3, size=(M, K)) * np.exp2(r.integers(-3, 4, size=(M, KS)).astype(float)).repeat(128, 1)[:, :K]
    w = r.integers(1, 3, size=(K, N)) * np.exp2(r.integers(-3, 4, size=(KS, N)).astype(float)).repeat(128, 0)[:K]
    Y, _ = run_linear(x, w, None)
    assert torch.equal(Y.cpu(), bf16(x @ w))      # sums below 2^24 units of 2^-6


def test_non_finite_rows_and_columns_stay_their_own():
    M, K, N = 70, 300 // 8 * 8, 200
    x, w = rand(1, M, K), rand(2, K, N, scale=0.05, loud=False)
    x[3, 7], x[69, 200] = np.inf, np.nan
    w[100, 11] = np.nan
    Y, _ = run_linear(x, w, None)
    nan = torch.isnan(Y.cpu()).numpy()
    want = np.zeros((M, N), bool)
    want[[3, 69]] = True
    want[:, 11] = True
    assert np.array_equal(nan, want)
    x[[3, 69]], w[:, 11] = 0, 0
    y, mag = fp8.linear(x, w)
    keep = ~want
    got = G.bf16_host(Y)
    assert (np.abs(got - y) <= 2.0 ** -8 * np.abs(y) + 2 * K * 2.0 ** -23 * mag)[keep].all()


@pytest.mark.parametrize("M,N", [(9, 200), (100, 200), (2600, 5640)])
@pytest.mark.parametrize("epilogue", EPI[1:])
def test_gelu_passes_nan_on_and_settles_far_out(M, N, epilogue):
    """NaN rows stay NaN through the GELUs; far out they are the value itself and zero."""
    K = 136
    x, w = np.zeros((M, K)), np.zeros((K, N))
    x[:, 0], w[0, 0::2], w[0, 1::2] = 64.0, 4.0, -4.0         # 256 and -256
    x[M - 1, 5] = np.nan
    Y, _ = run_linear(x, w, None, epilogue)
    got = G.bf16_host(Y)
    assert np.isnan(got[M - 1]).all()
    assert (got[:M - 1, 0::2] == 256).all() and (got[:M - 1, 1::2] == 0).all()


def test_zero_rows_give_the_bias():
    K, N = 256, 136
    w, b = rand(2, K, N, loud=False), rand(3, N, loud=False)
    Y, _ = run_linear(np.zeros((5, K)), w, b)
    assert torch.equal(Y.cpu(), bf16(b).expand(5, N))


def run_experts(x, w, offsets, b=None, epilogue=0, begin=0):
    E, K, N = w.shape
    ex = layer.FP8Experts(bf16(w).to(G.DEV), None if b is None else bf16(b).to(G.DEV), epilogue, begin)
    Y = G.poisoned_bf16(x.shape[0], N)
    ex(bf16(x).to(G.DEV), torch.tensor(offsets, dtype=torch.int32, device=G.DEV), Y)
    G.check_ok()
    return Y


@pytest.mark.parametrize("counts,tail", [
    ([1], 0), ([0, 3, 0, 0, 9, 1, 0], 0), ([0, 0, 0], 5), ([17, 0, 130, 1, 31, 8], 3), ([300, 5, 0, 77], 0),
    ([0] * 40 + [2] + [0] * 30 + [3], 1), ([7] * 33, 2), ([513, 1, 255, 0, 256], 11), ([1] * 100, 0), ([1500, 0, 257, 1, 2000, 903], 5)])
@pytest.mark.parametrize("epilogue", EPI)
def test_experts(counts, tail, epilogue):
    E, K, N = len(counts), 264, 136 if sum(counts) < 4000 else 5000     # the last: 256-row tiles on SM pairs
    T = sum(counts) + tail
    off = np.concatenate([[0], np.cumsum(counts)])
    x, w, b = rand(T, T, K), rand(E, E, K, N, scale=0.05, loud=False), rand(E + 1, E, N, loud=False)
    Y = run_experts(x, w, off.tolist(), b, epilogue, 50)
    want, mag = fp8.experts(x, w, off, b, epilogue, 50)
    live = ~np.isnan(want[:, 0])
    close(Y[torch.from_numpy(live).to(G.DEV)], want[live], mag[live], K, epilogue)
    assert torch.isnan(Y[torch.from_numpy(~live).to(G.DEV)]).all()      # as they were


def test_experts_that_start_behind_the_first_row():
    x, w = rand(1, 50, 128), rand(2, 2, 128, 64, scale=0.05, loud=False)
    Y = run_experts(x, w, [5, 21, 40])
    want, mag = fp8.experts(x, w, [5, 21, 40])
    live = ~np.isnan(want[:, 0])
    close(Y[torch.from_numpy(live).to(G.DEV)], want[live], mag[live], 128, 0)
    assert torch.isnan(Y[:5]).all() and torch.isnan(Y[40:]).all()


@pytest.mark.parametrize("offsets,taken", [
    ([-7, 10, 2 ** 31 - 1, 5], [0, 10, 40, 40]), ([0, 30, 20, 40], [0, 30, 30, 40]),
    ([2 ** 31 - 1, -2 ** 31, 0, 9], [40, 40, 40, 40]), ([3, 3, 3, 3], [3, 3, 3, 3])])
def test_offsets_that_break_the_rules_are_clamped(offsets, taken):
    """The kernel takes min(max(offset, 0), M), and no less than the offsets before: the rows that result are
    those of the clamped offsets, and nothing outside Y is written."""
    x, w = rand(1, 40, 128), rand(2, 3, 128, 64, scale=0.05, loud=False)
    Y = run_experts(x, w, offsets)
    want, mag = fp8.experts(x, w, taken)
    live = ~np.isnan(want[:, 0])
    close(Y[torch.from_numpy(live).to(G.DEV)], want[live], mag[live], 128, 0)
    assert torch.isnan(Y[torch.from_numpy(~live).to(G.DEV)]).all()


def test_512_experts():
    E, K, N = 512, 64, 24
    counts = np.random.default_rng(0).integers(0, 4, size=E)
    off = np.concatenate([[0], np.cumsum(counts)])
    x, w = rand(1, int(off[-1]), K), rand(2, E, K, N, scale=0.05, loud=False)
    Y = run_experts(x, w, off.tolist())
    close(Y, *fp8.experts(x, w, off), K, 0)


def test_host_built_layer_and_allocated_outputs():
    x, w = rand(1, 20, 128), rand(2, 128, 64, scale=0.05, loud=False)
    bits = bf16(w).view(torch.int16).numpy().view(np.uint16)
    Y = layer.FP8Linear.from_weight(bits)(bf16(x).to(G.DEV))
    close(Y, *fp8.linear(x, w), 128, 0)
    E = layer.FP8Experts.from_weight(bits[None])
    off = torch.tensor([0, 20], dtype=torch.int32, device=G.DEV)
    assert torch.equal(E(bf16(x).to(G.DEV), off), Y)
    part = E(bf16(x).to(G.DEV), off // 2)
    assert torch.equal(part[:10], Y[:10]) and (part[10:] == 0).all()


def test_weight_views():
    """A transposed weight and one expert of many, strided."""
    w = bf16(rand(1, 3, 136, 72, loud=False)).to(G.DEV)
    X = bf16(rand(2, 9, 136)).to(G.DEV)
    base = layer.FP8Linear(w[1].contiguous())(X)
    assert torch.equal(layer.FP8Linear(w[1].T.contiguous().T)(X), base)
    wide = torch.zeros(136, 100, dtype=torch.bfloat16, device=G.DEV)
    wide[:, 13:85] = w[1]
    assert torch.equal(layer.FP8Linear(wide[:, 13:85])(X), base)     # an odd first column: any bf16 alignment
    pair = layer.FP8Experts(w[::2])
    off = torch.tensor([0, 4, 9], dtype=torch.int32, device=G.DEV)
    Y = pair(X, off)
    assert torch.equal(Y[:4], layer.FP8Linear(w[0])(X)[:4]) and torch.equal(Y[4:], layer.FP8Linear(w[2])(X)[4:])


def test_layers_refuse():
    w = torch.zeros(64, 64, dtype=torch.bfloat16, device=G.DEV)
    lin, ex = layer.FP8Linear(w), layer.FP8Experts(w[None])
    X = torch.zeros(4, 64, dtype=torch.bfloat16, device=G.DEV)
    off = torch.tensor([0, 4], dtype=torch.int32, device=G.DEV)
    bad = [lambda: lin(X.float()), lambda: lin(X[:, :32]), lambda: lin(X.cpu()), lambda: lin(X[0]),
           lambda: lin(torch.zeros(64, 4, dtype=torch.bfloat16, device=G.DEV).T),
           lambda: lin(X, X[:2]), lambda: lin(X, X.float()), lambda: ex(X, off.long()), lambda: ex(X, off[:1]),
           lambda: ex(X, off.cpu()), lambda: ex(X, torch.zeros(4, dtype=torch.int32, device=G.DEV)[::2]),
           lambda: layer.FP8Linear(w.float()), lambda: layer.FP8Linear(w, w[0].float()), lambda: layer.FP8Linear(w, w[0][:8]),
           lambda: layer.FP8Linear(w, epilogue=9), lambda: layer.FP8Linear(w, gelu_col_begin=65)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: lin(X.expand(4, 64)[:1].expand(4, 64)), lambda: lin(X[:0]),
                 lambda: lin(torch.zeros(4, 68, dtype=torch.bfloat16, device=G.DEV)[:, 4:]),
                 lambda: layer.FP8Linear(w[:60])):
        with pytest.raises(lib.SvdqError):
            call()


def test_misaligned_bias_and_rows_that_interleave():
    K, N = 136, 264
    W, b = (bf16(rand(seed, *shape)).to(G.DEV) for seed, shape in ((1, (K, N)), (2, (N,))))
    off = torch.zeros(N + 3, dtype=torch.bfloat16, device=G.DEV)
    off[3:] = b
    fc, want = layer.FP8Linear(W, off[3:]), layer.FP8Linear(W, b)
    for M in (5, 77, 300):
        X = bf16(rand(M, M, K)).to(G.DEV)
        both = G.poisoned_bf16(M, K + N + 8)
        both[:, :K] = X
        fc(both[:, :K], Y=both[:, K:K + N])
        assert torch.equal(both[:, K:K + N], want(X)) and torch.equal(both[:, :K], X)
        assert torch.isnan(both[:, K + N:]).all()
        with pytest.raises(lib.SvdqError):
            fc(both[:, :K], Y=both[:, 8:8 + N])
    G.check_ok()


def test_two_streams_and_two_graphs_share_a_layer():
    """Calls of one instance that overlap on two streams, and two captured graphs replayed at once, have
    workspaces of their own."""
    K, N = 512, 1024
    lin = layer.FP8Linear(bf16(rand(1, K, N, scale=0.05, loud=False)).to(G.DEV))
    xs = [bf16(rand(10 + i, 900, K)).to(G.DEV) for i in range(2)]
    want = [lin(x).clone() for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [lin(x, stream=s) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs = [], []
    for x, s in zip(xs, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(lin(x))
        graphs.append(g)
    for _ in range(5):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    x0 = bf16(rand(20, 900, K)).to(G.DEV)
    xs[0].copy_(x0)                       # a replay reads its inputs anew
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], lin(x0)) and not torch.equal(outs[0], want[0])
    G.check_ok()


def test_offsets_from_the_kernel_before():
    """Offsets written on the device right before the call, and rewritten between replays of a graph."""
    E, K, N, T = 6, 256, 136, 200
    w = rand(1, E, K, N, scale=0.05, loud=False)
    ex = layer.FP8Experts(bf16(w).to(G.DEV))
    x = rand(2, T, K)
    X = bf16(x).to(G.DEV)
    route = torch.randint(0, E, (T,), device=G.DEV)
    Y = G.poisoned_bf16(T, N)
    ends = torch.arange(E, device=G.DEV)

    def step():
        off = torch.zeros(E + 1, dtype=torch.int32, device=G.DEV)
        off[1:] = (route[:, None] <= ends).sum(0)
        return ex(X, off, Y), off
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _, off = step()
    for seed in range(3):
        torch.manual_seed(seed)
        route.copy_(torch.randint(0, E, (T,), device=G.DEV))
        g.replay()
        torch.cuda.synchronize()
        o = off.tolist()
        assert o[-1] == T
        close(Y, *fp8.experts(x, w, o), K, 0)
    G.check_ok()


def test_repeats_are_bit_identical():
    x = bf16(rand(1, 333, 1000)).to(G.DEV)
    for m, n in ((1, 520), (20, 520), (333, 520), (333, 33000)):
        lin = layer.FP8Linear(bf16(rand(2, 1000, n, scale=0.05, loud=False)).to(G.DEV))
        first = lin(x[:m])
        for _ in range(10):
            assert torch.equal(lin(x[:m]), first)


def test_offsets_past_32_bits():
    """X and Y past 2^31 bytes, sampled rows on both sides."""
    M, K, N = 70000, 16384, 16392
    base = bf16(rand(1, 64, K)).to(G.DEV)
    X = base.repeat(M // 64 + 1, 1)[:M]
    w = rand(2, K, 8, scale=0.02, loud=False)
    W = torch.zeros(K, N, dtype=torch.bfloat16, device=G.DEV)
    W[:, :8] = bf16(w).to(G.DEV)
    W[:, -8:] = W[:, :8]
    Y = layer.FP8Linear(W)(X)
    G.check_ok()
    rows = [0, 63, 64, 65535, 65536, 65551, M - 1]
    assert rows[-1] * K * 2 > 2 ** 31 and rows[-1] * N * 2 > 2 ** 31
    x = base.double().cpu().numpy()[[r % 64 for r in rows]]
    want, mag = fp8.linear(x, w)
    close(Y[rows][:, :8], want, mag, K, 0)
    close(Y[rows][:, -8:], want, mag, K, 0)
    assert (Y[rows][:, 8:-8] == 0).all()


def test_block_of_layers():
    """The operators as a transformer block uses them: FP8 query, key and value projection, normed and turned
    heads, attention, FP8 output projection, and an MLP by expert, each against the oracle on the same bf16
    inputs; then the whole block captured in a graph, equal bit for bit."""
    T, H, D, E = 150, 4, 64, 5
    W = H * D
    wq, bq = rand(1, W, 3 * W, scale=0.05, loud=False), rand(2, 3 * W, scale=0.1, loud=False)
    wo = rand(3, W, W, scale=0.05, loud=False)
    w1, b1 = rand(4, E, W, 4 * W, scale=0.05, loud=False), rand(5, E, 4 * W, scale=0.1, loud=False)
    w2 = rand(6, E, 4 * W, W, scale=0.05, loud=False)
    dev = lambda a: bf16(a).to(G.DEV)
    qkv, out = layer.FP8Linear(dev(wq), dev(bq)), layer.FP8Linear(dev(wo))
    fc1, fc2 = layer.FP8Experts(dev(w1), dev(b1), lib.EPILOGUE_GELU_TANH), layer.FP8Experts(dev(w2))
    nq, nk = 1 + rand(7, D, scale=0.1, loud=False), 1 + rand(8, D, scale=0.1, loud=False)
    turn = layer.RotaryND([16, 24, 24], q_norm=dev(nq), k_norm=dev(nk))
    pos = torch.stack([torch.zeros(T), torch.arange(T) // 15, torch.arange(T) % 15], 1).to(torch.int32).to(G.DEV)
    counts = torch.tensor([0, 60, 1, 64, 25])
    off = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(torch.int32).to(G.DEV)
    order = torch.randperm(T, generator=torch.Generator().manual_seed(0)).to(G.DEV)
    X = dev(rand(9, T, W))

    def block(x):
        h = qkv(x)
        heads = h.unflatten(1, (3, H, D))
        q, k = turn(heads[:, 0], heads[:, 1], pos)
        a = torch.softmax(torch.einsum("mhd,nhd->hmn", q.float(), k.float()) / D ** 0.5, -1)
        o = torch.einsum("hmn,nhd->mhd", a, heads[:, 2].float()).reshape(T, W).to(torch.bfloat16)
        p = out(o)
        u = fc1(p[order], off)
        return h, q, k, o, p, u, fc2(u, off)

    h, q, k, o, p, u, y = block(X)
    torch.cuda.synchronize()
    G.check_ok()
    f = lambda t: t.double().cpu().numpy()
    close(h, *fp8.linear(f(X), wq, bq), W, 0)
    hh = f(h).reshape(T, 3, H, D)
    for got, i, n in ((q, 0, nq), (k, 1, nk)):
        want = rope.rope(hh[:, i], pos.cpu().numpy(), [16, 24, 24], w=bf16(n).double().numpy())
        assert (np.abs(f(got) - want) <= 2.0 ** -8 * np.abs(want) + 1e-5 * np.abs(want).max()).all()
    close(p, *fp8.linear(f(o), wo), W, 0)
    offs = off.cpu().numpy()
    close(u, *fp8.experts(f(p[order]), w1, offs, b1, 2), W, 2)
    close(y, *fp8.experts(f(u), w2, offs), 4 * W, 0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        again = block(X)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, (h, q, k, o, p, u, y)))


def gelu_sweep(N):
    """N bf16 values: every one of 2^-8 <= |b| <= 13 on the negative side and <= 8 on the other, over and over."""
    bits = torch.arange(0x3B80, 0x4151, dtype=torch.int16).view(torch.bfloat16)
    every = torch.cat([-bits, bits[bits <= 8]])
    return every.repeat(-(-N // len(every)))[:N]


def close_gelu(got, y):
    """GELU (erf) of exact arguments.  For y < 0 the result is y Phi(y), relative to which the kernel's polynomial for log2 Phi,
    evaluated in float32 on a dense grid, is off by less than 6.1e-6 down to -2, 4.8e-5 down to -5 and 4.1e-4 down to -13, and
    the exponential by 2^-22: 2^-17, 2^-14 and 2^-11 hold their sums.  For y >= 0 the result is y - y Phi(-y), of which no
    more than half is subtracted: 2^-17.  Then bf16's half step; below 2^-121 Phi itself is no normal float32 and may count
    as zero."""
    got, want = G.bf16_host(got), fp8.gelu(y, 1)
    rel = np.where(y >= -2, 2.0 ** -17, np.where(y >= -5, 2.0 ** -14, 2.0 ** -11))
    bad = ~(np.abs(got - want) <= (2.0 ** -8 + 1.01 * rel) * np.abs(want) + 2.0 ** -121)
    assert not bad.any(), (int(bad.sum()), y[bad][:6], got[bad][:6], want[bad][:6])


@pytest.mark.parametrize("M,K,N", [(3, 136, 2992), (40, 136, 2992), (140, 136, 2992), (2600, 2056, 5640)])
def test_gelu_erf_of_exact_arguments(M, K, N):
    """Arguments that are exact in float32: a bias of every bf16 value beside one product, of a row's own.  The last size
    takes the 256-row tiles."""
    b = gelu_sweep(N)
    shift = torch.arange(M) % 16 / 512                             # e4m3 values, exact beside any bias in 24 bits
    X, W = torch.zeros(M, K, dtype=torch.bfloat16), torch.zeros(K, N, dtype=torch.bfloat16)
    X[:, 5], W[5] = shift.to(torch.bfloat16), 1
    Y = layer.FP8Linear(W.to(G.DEV), b.to(G.DEV), lib.EPILOGUE_GELU_ERF)(X.to(G.DEV))
    G.check_ok()
    rows = sorted({*range(min(M, 16)), M // 2, M - 1})
    close_gelu(Y[rows], shift.double().numpy()[rows, None] + b.double().numpy())


@pytest.mark.parametrize("M", [1, 16, 40, 300])
def test_library_calls_equal_the_layers(M):
    """fp8_pack_weights, fp8_linear and fp8_linear_grouped by their bindings, with workspaces of the caller's."""
    K, N, E = 264, 136, 2
    w, b = bf16(rand(1, E, K, N, scale=0.05, loud=False)).to(G.DEV), bf16(rand(2, E, N, loud=False)).to(G.DEV)
    x = bf16(rand(3, M, K + 8)).to(G.DEV)[:, :K]
    need = lib.fp8_workspace_size(M, K)
    ws = G.poisoned_u8(need) if need else None
    Y = G.poisoned_bf16(M + 1, N + 8)
    lib.fp8_linear(x, lib.fp8_pack_weights(w[0]), b[0], N, lib.EPILOGUE_GELU_TANH, 40, Y[:M, :N], workspace=ws)
    assert torch.equal(Y[:M, :N], layer.FP8Linear(w[0], b[0], lib.EPILOGUE_GELU_TANH, 40)(x))
    assert torch.isnan(Y[M]).all() and torch.isnan(Y[:, N:]).all()
    need = lib.fp8_workspace_size(M, K, E)
    ws = G.poisoned_u8(need) if need else None
    packed = G.poisoned_u8(lib.fp8_weight_size(K, N, E) + 16)
    assert lib.fp8_pack_weights(w, packed[:-16]) is not None and (packed[-16:] == G.POISON).all()
    off = torch.tensor([0, M // 3, M], dtype=torch.int32, device=G.DEV)
    Y = G.poisoned_bf16(M + 1, N)
    lib.fp8_linear_grouped(x, off, packed, b, N, lib.EPILOGUE_NONE, 0, Y[:M], workspace=ws)
    assert torch.equal(Y[:M], layer.FP8Experts(w, b)(x, off)) and torch.isnan(Y[M]).all()
    G.check_ok()


def test_library_calls_refuse():
    M, K, N = 40, 264, 136
    w, x = (torch.zeros(*s, dtype=torch.bfloat16, device=G.DEV) for s in ((K, N), (M, K)))
    packed, ws = lib.fp8_pack_weights(w), G.poisoned_u8(lib.fp8_workspace_size(M, K))
    Y, off = G.poisoned_bf16(M, N), torch.tensor([0, M], dtype=torch.int32, device=G.DEV)
    b = torch.zeros(N, dtype=torch.bfloat16, device=G.DEV)
    lin = lambda x=x, p=packed, b=b, Y=Y, ws=ws: lib.fp8_linear(x, p, b, N, 0, 0, Y, workspace=ws)
    ex = lambda off=off, b=b, Y=Y, ws=ws: lib.fp8_linear_grouped(x, off, packed, b, N, 0, 0, Y, workspace=ws)
    for call in (lambda: lin(ws=None), lambda: lin(ws=ws[:-1]), lambda: lin(p=packed[:-1]), lambda: lin(b=b[:-1]),
                 lambda: lin(Y=Y[:-1]), lambda: lin(Y=Y[:, :-8]), lambda: lin(x=x.float()), lambda: lin(x=x.cpu()),
                 lambda: lin(x=torch.zeros(K, M, dtype=torch.bfloat16, device=G.DEV).T), lambda: lin(b=b.float()),
                 lambda: ex(ws=None), lambda: ex(off=off.long()), lambda: ex(off=off.cpu()), lambda: ex(b=b[:-1]),
                 lambda: ex(off=off[:, None]), lambda: ex(Y=Y[:-1]),
                 lambda: ex(off=torch.zeros(4, dtype=torch.int32, device=G.DEV)[::2])):
        with pytest.raises(ValueError):
            call()
    assert torch.isnan(Y).all()


# Few column tiles and a long K: the few-row kernel splits K over clusters of 2 (from 8 blocks of 128 on), 4 (16) and 8 (32)
# CTAs, here with an odd number of two-block stages and a last stage of one block as well.
SPLIT_K = [1024, 1032, 2048, 2184, 4096, 4104, 4352, 5000]


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 20, 32, 50, 64, 100, 128])
@pytest.mark.parametrize("N", [8, 136, 512])
def test_long_k_split_over_clusters(M, N):
    r = np.random.default_rng(M + N)
    for K in SPLIT_K:
        x, w = r.integers(-8, 9, size=(M, K)).astype(float), r.integers(-8, 9, size=(K, N)).astype(float)
        b = r.integers(-100, 101, size=N).astype(float)
        Y, Yf = run_linear(x, w, b, ldy=N + 8)
        assert torch.equal(Y.cpu(), bf16(x @ w + b)), K            # exact sums below 2^24
        assert torch.isnan(Yf[:, N:]).all(), K


@pytest.mark.parametrize("M", [1, 16, 20, 50, 100])
@pytest.mark.parametrize("K,epilogue", [(1032, 2), (2184, 1), (4104, 0), (4104, 1)])
def test_long_k_split_against_oracle_and_repeats(M, K, epilogue):
    N = 264
    x, w, b = rand(M, M, K), rand(K, K, N, scale=0.02, loud=False), rand(N, N, loud=False)
    want, mag = fp8.linear(x, w, b, epilogue, 100)
    lin = layer.FP8Linear(bf16(w).to(G.DEV), bf16(b).to(G.DEV), epilogue, 100)
    X = bf16(x).to(G.DEV)
    Y = lin(X)
    close(Y, want, mag, K, epilogue)
    for _ in range(5):
        assert torch.equal(lin(X), Y)
    G.check_ok()


@pytest.mark.parametrize("counts,start,tail", [
    ([0, 2, 0, 3], 1, 2), ([1], 0, 0), ([0, 0, 0], 2, 3), ([5, 0, 0, 0, 0, 0], 0, 0),     # 16-row tiles, X quantized inside
    ([3, 17], 0, 0), ([0, 19], 1, 0), ([13, 40], 2, 1), ([30, 60], 0, 5), ([0, 100], 3, 0)])
@pytest.mark.parametrize("N", [8, 200])
def test_experts_with_a_long_k(counts, start, tail, N):
    """Splits by expert: clusters without a unit of work (empty experts, rows of no expert), tiles that begin behind a
    multiple of 8 rows, repeats bit for bit."""
    r = np.random.default_rng(sum(counts) + N)
    E, T = len(counts), start + sum(counts) + tail
    off = start + np.concatenate([[0], np.cumsum(counts)])
    live = np.zeros(T, bool)
    live[off[0]:off[-1]] = True
    for K in (1032, 2048, 4104, 4352):
        x, w = r.integers(-8, 9, size=(T, K)).astype(float), r.integers(-8, 9, size=(E, K, N)).astype(float)
        b = r.integers(-100, 101, size=(E, N)).astype(float)
        Y = run_experts(x, w, off.tolist(), b)
        want = np.full((T, N), np.nan)
        for e in range(E):
            want[off[e]:off[e + 1]] = x[off[e]:off[e + 1]] @ w[e] + b[e]
        assert torch.equal(Y.cpu()[live], bf16(want[live])) and torch.isnan(Y.cpu()[~live]).all(), K
        again = run_experts(x, w, off.tolist(), b)
        assert torch.equal(again[live], Y[live])


@pytest.mark.parametrize("counts,start,tail", [([1500, 0, 257, 1, 2000, 903], 0, 5), ([0, 700, 9, 2500, 1101], 13, 40)])
def test_experts_on_the_256_row_tiles(counts, start, tail):
    """Rows enough, and a K long enough, for the SM pairs: ragged and empty experts, first rows that are no multiple of 8,
    bias rows of their own, exact sums."""
    g = torch.Generator(device=G.DEV).manual_seed(sum(counts))
    E, T, K, N = len(counts), start + sum(counts) + tail, 2056, 5000
    ints = lambda *s: torch.randint(-8, 9, s, generator=g, device=G.DEV).to(torch.bfloat16)
    x, w, b = ints(T, K), ints(E, K, N), ints(E, N)
    off = start + np.concatenate([[0], np.cumsum(counts)])
    Y = G.poisoned_bf16(T, N)
    ex = layer.FP8Experts(w, b)
    ex(x, torch.tensor(off, dtype=torch.int32, device=G.DEV), Y)
    G.check_ok()
    for e in range(E):
        rows = slice(int(off[e]), int(off[e + 1]))
        assert torch.equal(Y[rows], (x[rows].double() @ w[e].double() + b[e].double()).to(torch.bfloat16)), e
    assert torch.isnan(Y[:off[0]]).all() and torch.isnan(Y[off[-1]:]).all()


@pytest.mark.parametrize("epilogue", EPI[1:])
def test_gelu_of_experts_on_the_256_row_tiles(epilogue):
    """Each expert's own bias row and a column where the GELU begins, inside a run of 16 columns, on the SM pairs."""
    counts, K, N, begin = [1500, 0, 257, 1, 2000, 903], 2056, 5000, 1003
    E, T = len(counts), sum(counts)
    b = torch.stack([gelu_sweep(N).roll(100 * e) for e in range(E)])
    x, w = torch.zeros(T, K, dtype=torch.bfloat16), torch.zeros(E, K, N, dtype=torch.bfloat16)
    x[:, 7], w[:, 7] = (torch.arange(T) % 16 / 512).to(torch.bfloat16), 1
    off = np.concatenate([[0], np.cumsum(counts)])
    Y = G.poisoned_bf16(T, N)
    layer.FP8Experts(w.to(G.DEV), b.to(G.DEV), epilogue, begin)(
        x.to(G.DEV), torch.tensor(off, dtype=torch.int32, device=G.DEV), Y)
    G.check_ok()
    for row in (0, 1, 1499, 1500, 1756, 1757, 1758, 3757, 3758, T - 1):
        e = int(np.searchsorted(off, row, side="right")) - 1
        y = float(x[row, 7]) + b[e].double().numpy()
        assert torch.equal(Y[row, :begin].cpu(), torch.from_numpy(y[:begin]).to(torch.bfloat16)), row
        if epilogue == lib.EPILOGUE_GELU_ERF:
            close_gelu(Y[row:row + 1, begin:], y[None, begin:])
        else:
            close(Y[row:row + 1, begin:], fp8.gelu(y[None, begin:], 2), np.abs(y[None, begin:]), K, 2)


@pytest.mark.parametrize("epilogue", EPI[1:])
def test_gelu_and_nan_on_the_256_row_tiles(epilogue):
    M, K, N = 2600, 2056, 5640
    x, w = np.zeros((M, K)), np.zeros((K, N))
    x[:, 0], w[0, 0::2], w[0, 1::2] = 64.0, 4.0, -4.0         # 256 and -256
    x[M - 1, 5], x[300, 2000] = np.nan, np.inf
    Y, Yf = run_linear(x, w, None, epilogue, ldy=N + 8)
    bad = [300, M - 1]
    assert torch.isnan(Y[bad]).all() and torch.isnan(Yf[:, N:]).all()
    keep = torch.ones(M, dtype=torch.bool, device=G.DEV)
    keep[bad] = False
    assert (Y[keep][:, 0::2] == 256).all() and (Y[keep][:, 1::2] == 0).all()


@pytest.mark.parametrize("M,K,N", [(3, 136, 2992), (40, 136, 2992), (140, 136, 2992), (2600, 2056, 5640)])
def test_gelu_tanh_of_exact_arguments(M, K, N):
    """y / (1 + 2^x), x = -2 z log2 e: three float32 roundings of x (3 * 2^-24 |x| ln 2 of the exponential, |x| below 5.5 down
    to y = -2, 25 to -5, 134 further on), the exponential and the reciprocal 2^-22 each, sum and product 2^-24 each, are less
    than 2^-18, 2^-17 and 2^-15 of the result; the reciprocal is no normal float32 below 2^-121."""
    b = gelu_sweep(N)
    shift = torch.arange(M) % 16 / 512
    X, W = torch.zeros(M, K, dtype=torch.bfloat16), torch.zeros(K, N, dtype=torch.bfloat16)
    X[:, 5], W[5] = shift.to(torch.bfloat16), 1
    Y = layer.FP8Linear(W.to(G.DEV), b.to(G.DEV), lib.EPILOGUE_GELU_TANH)(X.to(G.DEV))
    G.check_ok()
    rows = sorted({*range(min(M, 16)), M // 2, M - 1})
    y = shift.double().numpy()[rows, None] + b.double().numpy()
    want = y / (1 + np.exp(-2 * np.sqrt(2 / np.pi) * (y + 0.044715 * y ** 3)))     # without 1 + tanh's cancellation
    rel = np.where(y >= -2, 2.0 ** -18, np.where(y >= -5, 2.0 ** -17, 2.0 ** -15))
    got = G.bf16_host(Y[rows])
    bad = ~(np.abs(got - want) <= (2.0 ** -8 + 1.01 * rel) * np.abs(want) + 2.0 ** -121)
    assert not bad.any(), (int(bad.sum()), y[bad][:6], got[bad][:6], want[bad][:6])
