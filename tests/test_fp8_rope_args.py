"""Refusals and size queries of the block-scaled FP8 calls and of rope_nd, without a GPU: every check happens
before anything touches the device."""
import ctypes

import pytest
import torch

from bit_w4a4_diffusion_smooth_b200 import layer, lib

P = ctypes.c_void_p(16)        # never dereferenced
ODD = ctypes.c_void_p(24)


def test_sizes():
    # K = 136: two stages, one scale word; 1001 rows take 1008; few rows an expert need no workspace
    assert lib.fp8_weight_size(136, 136, 3) == 3 * (136 * 2 * 128 + 2 * 512)
    assert lib.fp8_workspace_size(1001, 136) == 2 * 1008 * 128 + 1008 * 4
    assert lib.fp8_workspace_size(129, 8) == 136 * 128 + 136 * 4
    assert lib.fp8_workspace_size(16, 136) == lib.fp8_workspace_size(64, 136, 8) == 0
    assert lib.fp8_workspace_size(17, 136) > 0 and lib.fp8_workspace_size(65, 136, 8) > 0
    for bad in ((0, 8), (12, 8), (8, 0), (8, 12), (8, 8, 0), (8, 8, 513)):
        with pytest.raises(lib.SvdqError) as e:
            lib.fp8_weight_size(*bad)
        assert e.value.status == lib.ERR_SHAPE
    for bad in ((0, 8), (1, 4), (1, 0), (-1, 8), (2 ** 30 + 1, 8), (4, 8, 0), (4, 8, 513)):
        with pytest.raises(lib.SvdqError) as e:
            lib.fp8_workspace_size(*bad)
        assert e.value.status == lib.ERR_SHAPE


def _linear(x=P, M=4, K=64, ldx=64, w=P, bias=None, N=64, epi=0, begin=0, y=P, ldy=64, ws=P):
    return lib.load().fp8_linear(x, M, K, ldx, w, bias, N, epi, begin, y, ldy, ws, None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), lib.ERR_INVALID_ARG), (dict(w=None), lib.ERR_INVALID_ARG), (dict(y=None), lib.ERR_INVALID_ARG),
    (dict(M=129, ws=None), lib.ERR_INVALID_ARG), (dict(epi=3), lib.ERR_INVALID_ARG), (dict(epi=-1), lib.ERR_INVALID_ARG),
    (dict(M=0), lib.ERR_SHAPE), (dict(M=-5), lib.ERR_SHAPE), (dict(M=2 ** 30 + 1), lib.ERR_SHAPE), (dict(K=60), lib.ERR_SHAPE), (dict(K=0), lib.ERR_SHAPE),
    (dict(N=60), lib.ERR_SHAPE), (dict(N=0), lib.ERR_SHAPE), (dict(ldx=56), lib.ERR_SHAPE), (dict(ldx=68), lib.ERR_SHAPE),
    (dict(ldy=56), lib.ERR_SHAPE), (dict(ldy=68), lib.ERR_SHAPE), (dict(begin=-1), lib.ERR_SHAPE),
    (dict(begin=65), lib.ERR_SHAPE), (dict(M=2 ** 31 - 1, N=2 ** 20, ldy=2 ** 20), lib.ERR_SHAPE),
    (dict(x=ODD), lib.ERR_ALIGNMENT), (dict(w=ODD), lib.ERR_ALIGNMENT), (dict(y=ODD), lib.ERR_ALIGNMENT),
    (dict(M=129, ws=ODD), lib.ERR_ALIGNMENT), (dict(bias=ODD), lib.ERR_ALIGNMENT)])
def test_fp8_linear_refuses(kw, want):
    assert _linear(**kw) == want


def test_fp8_grouped_and_pack_refuse():
    so = lib.load()
    g = lambda off=P, E=2, M=4: so.fp8_linear_grouped(P, M, 64, 64, off, E, P, None, 64, 0, 0, P, 64, P, None)
    assert g(off=None) == lib.ERR_INVALID_ARG and g(off=ctypes.c_void_p(18)) == lib.ERR_ALIGNMENT
    assert g(E=0) == lib.ERR_SHAPE and g(E=513) == lib.ERR_SHAPE and g(M=0) == lib.ERR_SHAPE
    k = lambda W=P, K=64, N=64, ldw=64, st=0, E=1, out=P: so.fp8_pack_weights(W, K, N, ldw, st, E, out, None)
    assert k(W=None) == lib.ERR_INVALID_ARG and k(out=None) == lib.ERR_INVALID_ARG and k(out=ODD) == lib.ERR_ALIGNMENT
    assert k(K=4) == lib.ERR_SHAPE and k(N=4) == lib.ERR_SHAPE and k(ldw=63) == lib.ERR_SHAPE
    assert k(E=0) == lib.ERR_SHAPE and k(E=2, st=-1) == lib.ERR_SHAPE


def _plan(D=16, axes=2, pairing=0):
    p = lib.RopePlan(D, axes, pairing)
    for i in range(min(D // 2, 128)):
        p.axis[i], p.freq[i] = i % max(axes, 1), 1.0
    return p


def _rope(q=None, k=None, M=4, plan=None, pos=P, row=2, inverse=0):
    mk = lambda t: None if t is None else lib.ROPE_TENSOR.pack(*[0 if v is None else v for v in t])
    q = (16, 32, 16, 32, 32, 16, None, 2) if q is None else q
    plan = _plan() if plan is None else plan
    return lib.load().rope_nd(mk(q), mk(k), M, ctypes.byref(plan), pos, row, 0, inverse, 1e-6, None)


@pytest.mark.parametrize("kw,want", [
    (dict(pos=None), lib.ERR_INVALID_ARG), (dict(M=0), lib.ERR_SHAPE), (dict(M=2 ** 30 + 1), lib.ERR_SHAPE), (dict(row=-1), lib.ERR_SHAPE),
    (dict(plan=_plan(pairing=2)), lib.ERR_INVALID_ARG), (dict(plan=_plan(D=12)), lib.ERR_SHAPE),
    (dict(plan=_plan(D=264)), lib.ERR_SHAPE), (dict(plan=_plan(D=0)), lib.ERR_SHAPE), (dict(plan=_plan(axes=0)), lib.ERR_SHAPE),
    (dict(plan=_plan(axes=9)), lib.ERR_SHAPE), (dict(pos=ctypes.c_void_p(18)), lib.ERR_ALIGNMENT),
    # X, x_row, x_head, Y, y_row, y_head, norm, heads
    (dict(q=(None, 32, 16, 32, 32, 16, None, 2)), lib.ERR_INVALID_ARG),
    (dict(q=(16, 32, 16, None, 32, 16, None, 2)), lib.ERR_INVALID_ARG),
    (dict(q=(24, 32, 16, 32, 32, 16, None, 2)), lib.ERR_ALIGNMENT),
    (dict(q=(16, 36, 16, 32, 32, 16, None, 2)), lib.ERR_ALIGNMENT),
    (dict(q=(16, 32, 16, 32, 32, 16, 24, 2)), lib.ERR_ALIGNMENT),
    (dict(q=(16, 32, 16, 32, 32, 16, None, 0)), lib.ERR_SHAPE),
    (dict(q=(16, 32, 16, 32, 24, 16, None, 2)), lib.ERR_SHAPE),      # rows of Y overlap
    (dict(q=(16, 32, 16, 32, 32, 8, None, 2)), lib.ERR_SHAPE),       # heads of Y overlap
    (dict(q=(16, 32, 16, 32, 16, 48, None, 2)), lib.ERR_SHAPE),      # head-major, 4 rows of 16 in 48
    (dict(q=(16, 32, 16, 16, 64, 16, None, 2)), lib.ERR_INVALID_ARG),  # in place with other strides
    (dict(q=(16, 32, 16, 32, 32, 16, 64, 2), inverse=1), lib.ERR_INVALID_ARG),
    (dict(k=(16, 32, 16, 32, 32, 16, 64, 2), inverse=1), lib.ERR_INVALID_ARG),
    (dict(k=(16, 32, 16, 24, 32, 16, None, 2)), lib.ERR_ALIGNMENT)])
def test_rope_refuses(kw, want):
    assert _rope(**kw) == want


@pytest.mark.parametrize("kw", [
    # bytes: rows of 64, 4 rows from 256 on: 256 .. 512; Y of the same rows, one element run in them
    dict(x=256, y=256), dict(x=256, y=256 + 48), dict(x=256, y=496), dict(x=496, y=256), dict(x=256, y=272, ldx=32, ldy=40),
    dict(x=256, y=256 + 32, ldx=40, ldy=40), dict(M=1, x=256, y=304), dict(x=256, y=256 + 64 + 16, ldx=64, ldy=64)])
def test_fp8_refuses_a_y_on_top_of_x(kw):
    kw = dict(dict(M=4, ldx=32, ldy=32), **kw)
    x, y = ctypes.c_void_p(kw.pop("x")), ctypes.c_void_p(kw.pop("y"))
    assert _linear(x=x, y=y, K=32, N=32, **kw) == lib.ERR_INVALID_ARG
    assert b"overlaps" in lib.load().svdq_last_error_string()


@pytest.mark.parametrize("kw", [
    # apart, or interleaved rows: past the check, refused only for want of a device
    dict(x=256, y=512), dict(x=512, y=256), dict(x=256, y=256 + 64, ldx=64, ldy=64), dict(x=320, y=256, ldx=64, ldy=64),
    dict(x=256, y=256 + 96, ldx=80, ldy=80), dict(M=1, x=256, y=320)])
def test_fp8_takes_a_y_beside_x(kw):
    kw = dict(dict(M=4, ldx=32, ldy=32), **kw)
    x, y = ctypes.c_void_p(kw.pop("x")), ctypes.c_void_p(kw.pop("y"))
    if torch.cuda.is_available():
        pytest.skip("the call would run")
    assert _linear(x=x, y=y, K=32, N=32, **kw) == lib.ERR_NOT_INITIALIZED


def _cells(X, row, head, heads, M, D=16):
    return {X // 2 + m * row + h * head + d for m in range(M) for h in range(heads) for d in range(D)}


def test_rope_refuses_shared_elements_and_only_those():
    """Every pair of layouts of one buffer against a count of the elements they share."""
    if torch.cuda.is_available():
        pytest.skip("the accepted calls would run")
    D, seen = 16, [0, 0]
    layouts = [(M, row, head, hq, hk) for M, row, head, hq, hk in (
        (3, 96, 16, 2, 2), (3, 96, 16, 4, 1), (2, 96, 32, 2, 1), (4, 16, 80, 2, 2), (1, 16, 48, 2, 1), (3, 48, 16, 1, 2))]
    for M, row, head, hq, hk in layouts:
        for a in range(0, 320, 8):
            for b in (0, 16, 40, 64, 128, 400):
                base = 4096
                qx, kx, qy, ky = base, base + 2 * a, base + 2 * 2000, base + 2 * (2000 + b)
                for q, k in (((qx, qy), (kx, ky)), ((qx, qx), (kx, kx)), ((qx, kx), (kx, qx)), ((qx, kx), (ky, ky)),
                             ((qx, qx), (kx, ky))):
                    c = [_cells(v, row, head, n, M) for v, n in ((q[0], hq), (q[1], hq), (k[0], hk), (k[1], hk))]
                    bad = (q[0] != q[1] and c[0] & c[1]) or (k[0] != k[1] and c[2] & c[3]) or c[0] & c[3] or \
                        c[2] & c[1] or c[1] & c[3]
                    rc = _rope(q=(q[0], row, head, q[1], row, head, None, hq),
                               k=(k[0], row, head, k[1], row, head, None, hk), M=M)
                    assert rc == (lib.ERR_INVALID_ARG if bad else lib.ERR_NOT_INITIALIZED), (M, row, head, hq, hk, q, k)
                    seen[not bad] += 1
    assert min(seen) > 500, seen
    assert _rope(q=(16, 32, 16, 4096, 32, 16, None, 2), k=(4096, 64, 16, 9999 * 16, 64, 16, None, 2)) == lib.ERR_INVALID_ARG


def test_rope_refuses_an_axis_that_pos_lacks():
    p = _plan()
    p.axis[3] = 2
    assert _rope(plan=p) == lib.ERR_SHAPE


def test_layers_refuse_host_tensors_and_bad_shapes():
    w = torch.zeros(64, 64, dtype=torch.bfloat16)
    for make in (lambda: layer.FP8Linear(w), lambda: layer.FP8Experts(w[None]), lambda: layer.FP8Linear(w[None]),
                 lambda: layer.RotaryND([16, 3], device="cpu"), lambda: layer.RotaryND([]),
                 lambda: layer.RotaryND([4]), lambda: layer.RotaryND([200, 64]), lambda: layer.RotaryND([16], theta=0)):
        with pytest.raises(ValueError):
            make()


def test_sizes_past_a_c_int_are_refused_not_cut_down():
    """2^32 + 4 rows would arrive as 4."""
    far = torch.empty_strided((2, 64), (2 ** 31, 1), dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError):
        lib._row_stride(far, 64)
    for n in (2 ** 31, 2 ** 32 + 4, -2 ** 31 - 1):
        with pytest.raises(ValueError):
            lib._c_int(n, "rows")
    assert lib._c_int(2 ** 31 - 1, "rows") == 2 ** 31 - 1


def _span(X, row, head, heads, M, D=16):
    c = _cells(X, row, head, heads, M, D)
    return min(c), max(c)


def test_rope_refuses_shared_elements_under_other_strides():
    """Tensors whose strides differ: what shares an element is refused, what lies in ranges of its own or beside the
    other in rows of one stride is taken."""
    if torch.cuda.is_available():
        pytest.skip("the accepted calls would run")
    M, seen = 3, {"shared": 0, "apart": 0, "beside": 0}
    layouts = [(96, 16, 2), (96, 32, 2), (64, 16, 4), (16, 48, 2), (32, 96, 2), (32, 128, 2), (0, 16, 2), (16, 0, 2),
               (96, 48, 1), (32, 16, 4)]
    for xrow, xhead, heads in layouts:
        for yrow, yhead, n in layouts:
            if (xrow, xhead) == (yrow, yhead) or n != heads or not (yrow >= 96 and yhead <= 32 or yhead >= 48 and yrow):
                continue
            for off in range(-400, 400, 8):
                X, Y = 4096, 4096 + 2 * off
                if X == Y:
                    continue
                x, y = _cells(X, xrow, xhead, heads, M), _cells(Y, yrow, yhead, heads, M)
                if len(y) != M * heads * 16:                    # a Y that overlaps itself is refused for that
                    continue
                rc = _rope(q=(X, xrow, xhead, Y, yrow, yhead, None, heads), M=M)
                (x0, x1), (y0, y1) = _span(X, xrow, xhead, heads, M), _span(Y, yrow, yhead, heads, M)
                if x & y:
                    seen["shared"] += 1
                    assert rc == lib.ERR_INVALID_ARG, (xrow, xhead, yrow, yhead, heads, off)
                elif x0 > y1 or y0 > x1:
                    seen["apart"] += 1
                    assert rc == lib.ERR_NOT_INITIALIZED, (xrow, xhead, yrow, yhead, heads, off)
                elif xrow == yrow and (y0 - x0) % xrow >= (heads - 1) * xhead + 16 and \
                        (y0 - x0) % xrow + (heads - 1) * yhead + 16 <= xrow:
                    seen["beside"] += 1
                    assert rc == lib.ERR_NOT_INITIALIZED, (xrow, xhead, yrow, yhead, heads, off)
    assert min(seen.values()) >= 10, seen


def test_rope_refuses_an_output_inside_the_projection_it_reads():
    """A contiguous output viewed at an offset into the fused projection's buffer: other strides, shared elements."""
    M, H, D, row = 6, 2, 16, 3 * 2 * 16
    fused, k = 4096, 4096 + 2 * H * D
    q = (fused, row, D, fused + 2 * row, H * D, D, None, H)
    assert _rope(q=q, k=(k, row, D, 65536, row, D, None, H), M=M) == lib.ERR_INVALID_ARG
    # the query's output on the keys, the keys' on the queries
    q = (fused, row, D, k + 2 * row, H * D, D, None, H)
    assert _rope(q=q, k=(k, row, D, 65536, row, D, None, H), M=M) == lib.ERR_INVALID_ARG
    # windows of rows that overlap one another, and an output on the last of them
    q = (4096, 32, 16, 65536, 96, 16, None, 6)
    assert _rope(q=q, k=(32768, 32, 16, 4096 + 2 * 112, 32, 16, None, 2), M=2) == lib.ERR_INVALID_ARG
    if not torch.cuda.is_available():
        # in place beside values between the key heads: other head strides in rows of one stride
        row = 8 * 16
        q = (4096, row, 16, 4096, row, 16, None, 4)
        kv = (4096 + 2 * 64, row, 32, 4096 + 2 * 64, row, 32, None, 2)
        assert _rope(q=q, k=kv, M=M) == lib.ERR_NOT_INITIALIZED
        # and the same by heads: planes of one stride, rows of others
        q = (4096, 16, 512, 4096, 16, 512, None, 2)
        kv = (4096 + 2 * 256, 32, 512, 4096 + 2 * 256, 32, 512, None, 2)
        assert _rope(q=q, k=kv, M=M) == lib.ERR_NOT_INITIALIZED


def _meta(shape, stride):
    return torch.empty_strided(shape, stride, dtype=torch.bfloat16, device="meta")


def test_layer_refuses_sizes_past_a_c_int():
    """The layer's own check, on tensors without memory: 2^31 rows, and row strides of 2^31 and 2^32 + 64."""
    lin = layer.FP8Linear.__new__(layer.FP8Linear)
    lin.K, lin.N, lin.device, lin.bias = 64, 64, torch.device("meta"), None
    ok = _meta((2, 64), (64, 1))
    for X, Y in ((_meta((2 ** 31, 64), (64, 1)), None), (_meta((2, 64), (2 ** 31, 1)), None),
                 (_meta((2, 64), (2 ** 32 + 64, 1)), None), (ok, _meta((2, 64), (2 ** 31, 1))),
                 (ok, _meta((2, 64), (2 ** 32 + 64, 1)))):
        with pytest.raises(ValueError, match="too large"):
            lin._call(X, None, Y, 0)


def test_library_calls_refuse_sizes_past_a_c_int():
    packed = torch.empty(lib.fp8_weight_size(64, 64), dtype=torch.uint8)
    many, wide = _meta((2 ** 31, 64), (64, 1)), _meta((2, 2 ** 32 + 64), (2 ** 32 + 64, 1))
    off = torch.zeros(2, dtype=torch.int32)
    for X in (many, wide):
        with pytest.raises(ValueError, match="too large"):
            lib.fp8_linear(X, packed, None, 64, 0, 0, X)
        with pytest.raises(ValueError, match="too large"):
            lib.fp8_linear_grouped(X, off, packed, None, 64, 0, 0, X)
    for W in (_meta((64, 2 ** 31), (2 ** 31, 1)), _meta((2 ** 32 + 64, 64), (64, 1))):
        with pytest.raises(ValueError, match="too large"):
            lib.fp8_pack_weights(W)
    with pytest.raises(ValueError):
        lib.fp8_pack_weights(W[0])
