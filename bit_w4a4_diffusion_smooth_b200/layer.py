"""User-facing layers on top of the C ABI: SVDQLinear (W4A4 + low-rank branch),
SVDQLinearInt4 (its INT4 variant), AWQLinear (W4A16), FP8Linear and FP8Experts (block-scaled FP8, dense and by
expert), and RotaryND (rotary positions over several axes).  They hold the packed weights on the GPU; all
arithmetic runs in the library.

The 4-bit layers keep one set of activation buffers per row count, shared by
all their calls: use such an instance from one stream at a time (two calls
with the same row count that overlap on different streams would race on them).
FP8Linear, FP8Experts and RotaryND keep nothing from one call for the next:
their workspaces and outputs come from torch's allocator, on the stream the
call runs on, so an instance may be used from several streams and captured
into several graphs.
"""
import numpy as np
import torch

from . import lib


def _resolve(device):
    """torch.device with an explicit index ('cuda' means the caller's current device)."""
    d = torch.device(device)
    if d.type != "cuda":
        raise ValueError(f"the layers run on a CUDA device, got {d}")
    return d if d.index is not None else torch.device("cuda", torch.cuda.current_device())


def _init_on(device):
    """svdq_init for `device` (it validates the GPU and makes it current), then restores the
    caller's current device."""
    prev = torch.cuda.current_device()
    try:
        lib.svdq_init(device.index)
    finally:
        torch.cuda.set_device(prev)


def _dev(a, device, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    if dtype is not None:
        t = t.view(dtype)
    return t.to(device)


def _check_input(X, K, device, name):
    if X.dim() != 2 or X.shape[1] != K:
        raise ValueError(f"{name}: X must be [M, {K}], got {tuple(X.shape)}")
    if X.dtype != torch.bfloat16 or X.device != device:
        raise ValueError(f"{name}: X must be bf16 on {device}, got {X.dtype} on {X.device}")


def _raw_stream(stream, device):
    """The CUDA stream handle a call enqueues on: `stream`, else the caller's current stream."""
    if stream is not None:
        return stream.cuda_stream
    get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return get(device.index) if get is not None else torch.cuda.current_stream(device).cuda_stream


class _Plans:
    """Marshalled C-ABI arguments of a layer's calls, per set of buffers.

    The key holds every property the checked path validates (pointers, shapes, strides and
    dtypes of X and Y, and the stream), so a hit repeats a call that already passed the
    checks with the same buffers; the library then finds its tensor maps cached as well.
    Bounded: the table is cleared when it fills."""

    LIMIT = 64

    def __init__(self):
        self._t = {}

    @staticmethod
    def key(X, Y, s):
        return (X.data_ptr(), X.shape[0], X.shape[1], X.stride(0), X.stride(1), X.dtype,
                Y.data_ptr(), Y.shape[0], Y.shape[1], Y.stride(0), Y.stride(1), Y.dtype, s)

    def get(self, k):
        return self._t.get(k)

    def put(self, k, plan):
        if len(self._t) >= self.LIMIT:
            self._t.clear()
        self._t[k] = plan


def _check_output(Y, M, N, device, name):
    if tuple(Y.shape) != (M, N) or Y.dtype != torch.bfloat16 or Y.device != device:
        raise ValueError(f"{name}: Y must be bf16 [{M}, {N}] on {device}, got {Y.dtype} {tuple(Y.shape)} "
                         f"on {Y.device}")


class SVDQLinear:
    """Y = (X^ L1) L2 + Q(X^) Q(R) + b  (one SVDQuant linear layer).

    Build with `from_weight` (offline host pack of a bf16 weight [K, N] and
    calibration maxima) or with the constructor from a dict returned by
    lib.svdq_pack_weights.
    """

    def __init__(self, packed, K, N, rank, bias_bits=None, epilogue=lib.EPILOGUE_NONE, gelu_col_begin=0,
                 device="cuda"):
        self.K, self.N, self.rank = K, N, rank
        self.epilogue, self.gelu_col_begin = epilogue, gelu_col_begin
        self.device = _resolve(device)
        _init_on(self.device)
        device = self.device
        self.inv_lambda = _dev(packed["inv_lambda"], device)
        self.l1t = _dev(packed["l1t"], device, torch.bfloat16) if rank else None
        self.l2t = _dev(packed["l2t"], device)
        self.w_bundle = _dev(packed["w_bundle"], device)
        self.s_w = _dev(np.asarray(packed["s_w"], np.float32).reshape(1), device)
        self.s_a = _dev(np.asarray(packed["s_a"], np.float32).reshape(1), device)
        self.bias = _dev(bias_bits, device, torch.bfloat16) if bias_bits is not None else None
        if self.bias is not None and self.bias.numel() != N:
            raise ValueError(f"SVDQLinear: bias must have {N} elements")
        self._bufs = {}
        self._plans = _Plans()

    @classmethod
    def from_weight(cls, W_bits, act_absmax, rank, bias_bits=None, epilogue=lib.EPILOGUE_NONE,
                    gelu_col_begin=0, device="cuda", seed=0):
        K, N = W_bits.shape
        packed = lib.svdq_pack_weights(W_bits, act_absmax, rank, seed=seed)
        return cls(packed, K, N, rank, bias_bits, epilogue, gelu_col_begin, device)

    def buffers(self, M):
        """Activation-side buffers for M rows (allocated once per M, shared by every call)."""
        if M not in self._bufs:
            sz = lib.svdq_act_sizes(M, self.K)
            self._bufs[M] = dict(
                a_bundle=torch.empty(sz["a_bundle"], dtype=torch.uint8, device=self.device),
                U=torch.empty(sz["u"], dtype=torch.uint8, device=self.device))
        return self._bufs[M]

    def quantize(self, X, stream=None):
        _check_input(X, self.K, self.device, "SVDQLinear")
        b = self.buffers(X.shape[0])
        lib.svdq_quantize_act(X, self.inv_lambda, self.l1t, self.rank, self.s_a, self.s_w,
                              b["a_bundle"], b["U"], stream=stream)
        return b

    def gemm(self, b, M, Y, stream=None):
        _check_output(Y, M, self.N, self.device, "SVDQLinear")
        lib.svdq_linear_w4a4(b["a_bundle"], b["U"], self.s_a, self.w_bundle, self.l2t, self.s_w, self.bias,
                             M, self.N, self.K, self.rank, self.epilogue, self.gelu_col_begin, Y, stream=stream)
        return Y

    def __call__(self, X, Y=None, stream=None):
        _check_input(X, self.K, self.device, "SVDQLinear")
        M = X.shape[0]
        if Y is None:
            Y = torch.empty((M, self.N), dtype=torch.bfloat16, device=self.device)
        s = _raw_stream(stream, self.device)
        key = _Plans.key(X, Y, s)
        plan = self._plans.get(key)
        if plan is None:
            # first call with these buffers: the checked wrappers, then the marshalled arguments
            self.gemm(self.quantize(X, stream), M, Y, stream)
            b = self.buffers(M)
            p = lambda t: None if t is None else t.data_ptr()
            q = (p(X), M, self.K, X.stride(0), p(self.inv_lambda), p(self.l1t), self.rank, p(self.s_a),
                 p(self.s_w), p(b["a_bundle"]), p(b["U"]), s)
            g = (p(b["a_bundle"]), p(b["U"]), p(self.s_a), p(self.w_bundle), p(self.l2t), p(self.s_w), p(self.bias),
                 M, self.N, self.K, self.rank, self.epilogue, self.gelu_col_begin, p(Y), Y.stride(0), s)
            self._plans.put(key, (q, g))
            return Y
        L = lib.load()
        lib._check("svdq_quantize_act", L.svdq_quantize_act(*plan[0]))
        lib._check("svdq_linear_w4a4", L.svdq_linear_w4a4(*plan[1]))
        return Y


class SVDQLinearInt4:
    """The INT4 W4A4 variant of SVDQLinear: the same smoothing and low-rank branch, the 4-bit
    branch in INT4 groups of 64 along K with bf16 scales (svdq_quantize_act_int4 +
    svdq_linear_int4).

    Build with `from_weight` (host pack) or from a dict returned by lib.svdq_pack_weights_int4.
    N must be a multiple of 128 (a multiple of 256 runs on the tensor cores).
    """

    def __init__(self, packed, K, N, rank, bias_bits=None, epilogue=lib.EPILOGUE_NONE, gelu_col_begin=0,
                 device="cuda"):
        self.K, self.N, self.rank = K, N, rank
        self.epilogue, self.gelu_col_begin = epilogue, gelu_col_begin
        self.device = _resolve(device)
        _init_on(self.device)
        device = self.device
        self.inv_lambda = _dev(packed["inv_lambda"], device)
        self.l1t = _dev(packed["l1t"], device, torch.bfloat16) if rank else None
        self.l2t = _dev(packed["l2t"], device)
        self.w_codes = _dev(packed["w_codes"], device)
        self.w_scales = _dev(packed["w_scales"], device)
        self.bias = _dev(bias_bits, device, torch.bfloat16) if bias_bits is not None else None
        if self.bias is not None and self.bias.numel() != N:
            raise ValueError(f"SVDQLinearInt4: bias must have {N} elements")
        self._bufs = {}

    @classmethod
    def from_weight(cls, W_bits, act_absmax, rank, bias_bits=None, epilogue=lib.EPILOGUE_NONE,
                    gelu_col_begin=0, device="cuda", seed=0):
        K, N = W_bits.shape
        packed = lib.svdq_pack_weights_int4(W_bits, act_absmax, rank, seed=seed)
        return cls(packed, K, N, rank, bias_bits, epilogue, gelu_col_begin, device)

    def buffers(self, M):
        """Activation-side buffers for M rows (allocated once per M, shared by every call)."""
        if M not in self._bufs:
            sz = lib.svdq_int4_act_sizes(M, self.K)
            self._bufs[M] = dict(
                codes=torch.empty(sz["codes"], dtype=torch.uint8, device=self.device),
                scales=torch.empty(sz["scales"], dtype=torch.uint8, device=self.device),
                U=torch.empty(lib.svdq_act_sizes(M, self.K)["u"], dtype=torch.uint8, device=self.device))
        return self._bufs[M]

    def __call__(self, X, Y=None, stream=None):
        _check_input(X, self.K, self.device, "SVDQLinearInt4")
        M = X.shape[0]
        if Y is None:
            Y = torch.empty((M, self.N), dtype=torch.bfloat16, device=self.device)
        _check_output(Y, M, self.N, self.device, "SVDQLinearInt4")
        b = self.buffers(M)
        lib.svdq_quantize_act_int4(X, self.inv_lambda, self.l1t, self.rank, b["codes"], b["scales"], b["U"],
                                   stream=stream)
        lib.svdq_linear_int4(b["codes"], b["scales"], b["U"], self.w_codes, self.w_scales, self.l2t, self.bias, M,
                             self.N, self.K, self.rank, self.epilogue, self.gelu_col_begin, Y, stream=stream)
        return Y


class SplitProjection:
    """A fused projection's packed checkpoint mapped onto split modules.

    The pages note that a checkpoint whose query, key and value projections
    are fused into one grouped operation does not map by itself onto a model
    that keeps them as separate modules: the mapping needs the tensor order
    and a small runtime adapter.  This is that adapter for an SVDQLinear
    packed over the concatenation [W_0 | W_1 | ...] of the parts along N
    (in that order): every part keeps the fused layer's smoothing, L1, s_a
    and s_w, and takes its own columns of the residual codes and scales, of
    L2^T and of the bias - views of the fused layer's device buffers, no
    copy.  One call quantizes X once (the parts share the activation side)
    and runs the parts' GEMMs as one grouped launch; part i's output equals
    columns [n_i, n_i + size_i) of the fused layer's output bit for bit.
    Part sizes must be multiples of 256 (the weight bundle's tile rows).
    """

    def __init__(self, fused, sizes, names=None):
        if sum(sizes) != fused.N or any(sz <= 0 or sz % 256 for sz in sizes):
            raise ValueError(f"SplitProjection: part sizes {sizes} must be positive multiples of 256 adding up to "
                             f"N = {fused.N}")
        if len(sizes) > lib.MAX_GROUP:
            raise ValueError(f"SplitProjection: at most {lib.MAX_GROUP} parts")
        self.fused = fused
        self.names = list(names) if names is not None else [str(i) for i in range(len(sizes))]
        tile_bytes = lib.svdq_weight_sizes(fused.K, 256, fused.rank)["w_bundle"]   # one 256-row tile row, all K
        self.parts = []
        n0 = 0
        for sz in sizes:
            n1 = n0 + sz
            begin = min(max(fused.gelu_col_begin - n0, 0), sz)
            self.parts.append(dict(n0=n0, N=sz, gelu_col_begin=begin,
                                   w_bundle=fused.w_bundle[n0 // 256 * tile_bytes:n1 // 256 * tile_bytes],
                                   l2t=fused.l2t[n0 * 2 * lib.LR_STRIDE:n1 * 2 * lib.LR_STRIDE],
                                   bias=fused.bias[n0:n1] if fused.bias is not None else None))
            n0 = n1

    def __call__(self, X, out=None, stream=None):
        """X: bf16 CUDA [M, K] -> {name: Y_i bf16 [M, size_i]} (or into the tensors of `out`)."""
        f = self.fused
        M = X.shape[0]
        b = f.quantize(X, stream)
        ys = {}
        probs = []
        for name, p in zip(self.names, self.parts):
            Y = out[name] if out is not None else torch.empty((M, p["N"]), dtype=torch.bfloat16, device=f.device)
            _check_output(Y, M, p["N"], f.device, "SplitProjection")
            ys[name] = Y
            probs.append(dict(a_bundle=b["a_bundle"], U=b["U"], s_a=f.s_a, w_bundle=p["w_bundle"], l2t=p["l2t"],
                              s_w=f.s_w, bias=p["bias"], M=M, N=p["N"], K=f.K, gelu_col_begin=p["gelu_col_begin"],
                              Y=Y))
        lib.svdq_linear_w4a4_grouped(probs, f.rank, f.epilogue, stream=stream)
        return ys


class AWQLinear:
    """Y = (X diag(inv_awq)) deq(W_a) + b with 4-bit group-64 weights, any M.

    Up to `gemm_rows` rows run on the GEMV (one pass over the packed weights per
    block of 16 rows); more rows run the GEMM path on weights expanded once into
    a workspace the layer keeps (allocated on first use, grown with M).
    """

    gemm_rows = 48

    def __init__(self, packed, K, N, bias_bits=None, device="cuda"):
        self.K, self.N = K, N
        self.device = _resolve(device)
        _init_on(self.device)
        device = self.device
        self.qweight = _dev(packed["qweight"], device)
        self.scales = _dev(packed["scales"], device, torch.bfloat16)
        self.zeros = _dev(packed["zeros"], device, torch.bfloat16)
        self.inv_awq = _dev(packed["inv_awq"], device)
        self.bias = _dev(bias_bits, device, torch.bfloat16) if bias_bits is not None else None
        if self.bias is not None and self.bias.numel() != N:
            raise ValueError(f"AWQLinear: bias must have {N} elements")

    @classmethod
    def from_weight(cls, W_bits, awq_scale, bias_bits=None, device="cuda"):
        K, N = W_bits.shape
        return cls(lib.awq_pack_weights(W_bits, awq_scale), K, N, bias_bits, device)

    def __call__(self, X, Y=None, stream=None):
        _check_input(X, self.K, self.device, "AWQLinear")
        if Y is None:
            Y = torch.empty((X.shape[0], self.N), dtype=torch.bfloat16, device=self.device)
        _check_output(Y, X.shape[0], self.N, self.device, "AWQLinear")
        if X.shape[0] > self.gemm_rows:
            need = lib.awq_gemm_workspace_size(X.shape[0], self.K, self.N)
            if getattr(self, "_workspace", None) is None or self._workspace.numel() < need:
                # (re)allocated: the expanded weights are written once into its head and reused
                self._workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
                lib.awq_expand_weights(self.inv_awq, self.qweight, self.scales, self.zeros, self.K, self.N,
                                       self._workspace, stream=stream)
            lib.awq_linear_w4a16_expanded(X, self.bias, self.N, Y, self._workspace, stream=stream)
        else:
            lib.awq_linear_w4a16(X, self.inv_awq, self.qweight, self.scales, self.zeros, self.bias, self.N, Y,
                                 stream=stream)
        return Y


# The caller's current device and its current stream's handle; torch's public functions for them take several times
# as long, which shows in calls whose GPU time is a few microseconds.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)


def _on(device, stream, call, *args):
    """call(*args, raw stream) with `device` current and torch allocating on the stream the work runs on: `stream`,
    else the caller's current stream of that device."""
    index = device.index
    if stream is None:
        if _current_device() == index:
            return call(*args, _current_stream(index))
        with torch.cuda.device(device):
            return call(*args, _current_stream(index))
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the layer on {device}")
    with torch.cuda.stream(stream):           # makes the stream's device current as well
        return call(*args, stream.cuda_stream)


def _aligned(t):
    """A vector as the kernels take it: contiguous, on a 16-byte boundary (`t` itself if it is)."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class FP8Linear:
    """Y = epilogue(q(X) q(W) + b) in block-scaled FP8: e4m3 codes under one power-of-two scale per 128 elements
    along K, for every row of X and every column of W (for projections that 4 bits lose too much of).

    weight: bf16 CUDA [K, N], quantized once here; bias: bf16 CUDA [N] or None.  `from_weight` takes the host
    arrays the other layers take.
    """

    experts = None

    def __init__(self, weight, bias=None, epilogue=lib.EPILOGUE_NONE, gelu_col_begin=0):
        name = type(self).__name__
        lead = () if self.experts is None else (self.experts,)
        if weight.dim() != len(lead) + 2 or weight.dtype != torch.bfloat16 or not weight.is_cuda:
            raise ValueError(f"{name}: weight must be a bf16 CUDA tensor {'[experts, K, N]' if lead else '[K, N]'}, "
                             f"got {weight.dtype} {tuple(weight.shape)} on {weight.device}")
        self.K, self.N = weight.shape[-2:]
        if epilogue not in (lib.EPILOGUE_NONE, lib.EPILOGUE_GELU_ERF, lib.EPILOGUE_GELU_TANH):
            raise ValueError(f"{name}: unknown epilogue {epilogue}")
        if not 0 <= gelu_col_begin <= self.N:
            raise ValueError(f"{name}: gelu_col_begin must be in [0, {self.N}]")
        self.epilogue, self.gelu_col_begin = epilogue, gelu_col_begin
        self.device = _resolve(weight.device)
        if bias is not None and (tuple(bias.shape) != (*lead, self.N) or bias.dtype != torch.bfloat16
                                 or bias.device != self.device):
            raise ValueError(f"{name}: bias must be bf16 {[*lead, self.N]} on {self.device}")
        _init_on(self.device)
        with torch.cuda.device(self.device):
            self.bias = None if bias is None else _aligned(bias)
            self.packed = lib.fp8_pack_weights(weight if weight.stride(-1) == 1 else weight.contiguous())
            torch.cuda.current_stream().synchronize()   # ready on every stream from here on

    @classmethod
    def from_weight(cls, W_bits, bias_bits=None, epilogue=lib.EPILOGUE_NONE, gelu_col_begin=0, device="cuda"):
        """From uint16 arrays of bf16 patterns on the host."""
        device = _resolve(device)
        bias = None if bias_bits is None else _dev(bias_bits, device, torch.bfloat16)
        return cls(_dev(W_bits, device, torch.bfloat16), bias, epilogue, gelu_col_begin)

    def _call(self, X, offsets, Y, s):
        """The checked call on raw stream `s`, which torch allocates on."""
        shape, K, N = X.shape, self.K, self.N
        if len(shape) != 2 or shape[1] != K or X.dtype is not torch.bfloat16 or X.get_device() != self.device.index:
            _check_input(X, K, self.device, type(self).__name__)   # says which
        M = shape[0]
        ldx, step = X.stride()
        if Y is None:
            Y, ldy = (X.new_empty(M, N) if offsets is None else X.new_zeros((M, N))), N
        else:
            _check_output(Y, M, N, self.device, type(self).__name__)
            ldy, y_step = Y.stride()
            step = step if y_step == 1 else 0
        if step != 1:
            raise ValueError(f"{type(self).__name__}: X and Y must have unit stride in their last dimension")
        if M == 1:                                # a single row's stride is its width, whatever torch recorded
            ldx, ldy = K, N
        elif M >= 2 ** 31 or ldx >= 2 ** 31 or ldy >= 2 ** 31:
            # a C int would cut these down without a word
            raise ValueError(f"{type(self).__name__}: X or Y is too large")
        experts = self.experts or 1
        need = lib.fp8_workspace_size(M, K, experts)
        ws = torch.empty(need, dtype=torch.uint8, device=self.device) if need else None
        bias = self.bias
        args = (self.packed.data_ptr(), None if bias is None else bias.data_ptr(), N, self.epilogue,
                self.gelu_col_begin, Y.data_ptr(), ldy, None if ws is None else ws.data_ptr(), s)
        L = lib.load()
        if offsets is None:
            rc = L.fp8_linear(X.data_ptr(), M, K, ldx, *args)
        else:
            rc = L.fp8_linear_grouped(X.data_ptr(), M, K, ldx, offsets.data_ptr(), experts, *args)
        if rc:
            lib._check("fp8_linear" if offsets is None else "fp8_linear_grouped", rc)
        return Y

    def __call__(self, X, Y=None, stream=None):
        """X: bf16 CUDA [M, K] -> bf16 [M, N] (into Y if given)."""
        return _on(self.device, stream, self._call, X, None, Y)


class FP8Experts(FP8Linear):
    """The FP8 product by expert: rows offsets[e] .. offsets[e+1]-1 of X meet weight e, any share of the rows.

    weight: bf16 CUDA [experts, K, N]; bias: bf16 CUDA [experts, N] or None.  `offsets` stay on the device (int32
    [experts + 1], not decreasing); rows of Y outside every expert's are left as they were.  A call that allocates Y
    fills it with zeros first, a pass over the whole output: 55 us more on 265 for 9216 rows x 10240, so give a Y
    where time counts.
    """

    def __init__(self, weight, bias=None, epilogue=lib.EPILOGUE_NONE, gelu_col_begin=0):
        self.experts = weight.shape[0] if weight.dim() == 3 else 0
        super().__init__(weight, bias, epilogue, gelu_col_begin)

    def __call__(self, X, offsets, Y=None, stream=None):
        if (offsets.dtype != torch.int32 or offsets.dim() != 1 or offsets.numel() != self.experts + 1
                or offsets.device != self.device or not offsets.is_contiguous()):
            raise ValueError(f"FP8Experts: offsets must be contiguous int32 [{self.experts + 1}] on {self.device}, got "
                             f"{offsets.dtype} {tuple(offsets.shape)} on {offsets.device}")
        return _on(self.device, stream, self._call, X, offsets, Y)


class RotaryND:
    """Rotary positions over several axes for query and key heads, after an optional RMS norm of each head.

    axis_dims: the share of the head dimension each axis turns (even, adding up to D); pair j of an axis of d
    dimensions turns by position * theta^(-2j/d).  interleaved: pairs are neighbours (2i, 2i+1), else i and
    i + D/2.  q_norm, k_norm: bf16 CUDA [D] norm weights or None.
    """

    def __init__(self, axis_dims, theta=10000.0, interleaved=True, q_norm=None, k_norm=None, eps=1e-6, device="cuda"):
        axis_dims = [int(d) for d in axis_dims]
        D = sum(axis_dims)
        if not axis_dims or any(d < 2 or d % 2 for d in axis_dims) or D % 8 or D > 256:
            raise ValueError(f"RotaryND: axis_dims {axis_dims} must be even and add up to a multiple of 8, at most 256")
        if not theta > 0:
            raise ValueError("RotaryND: theta must be positive")
        self.D, self.axes, self.eps = D, len(axis_dims), float(eps)
        self.device = _resolve(device)
        for w in (q_norm, k_norm):
            if w is not None and (w.dtype != torch.bfloat16 or w.numel() != D or w.device != self.device):
                raise ValueError(f"RotaryND: a norm weight must be bf16 [{D}] on {self.device}")
        _init_on(self.device)
        with torch.cuda.device(self.device):
            self.q_norm = None if q_norm is None else _aligned(q_norm)
            self.k_norm = None if k_norm is None else _aligned(k_norm)
            torch.cuda.current_stream().synchronize()   # ready on every stream from here on
        pairs = [(a, float(theta) ** (-2.0 * j / d)) for a, d in enumerate(axis_dims) for j in range(d // 2)]
        self.plan = lib.RopePlan(D, self.axes, lib.ROPE_ND_INTERLEAVED if interleaved else lib.ROPE_ND_HALF)
        for i, (a, f) in enumerate(pairs):
            self.plan.axis[i], self.plan.freq[i] = a, f

    def __call__(self, q, k, pos, q_out=None, k_out=None, inverse=False, stream=None):
        """q: bf16 CUDA [M, heads, D] (any row and head strides), k likewise or None; pos: int32 or float32
        [M, axes].  Returns (q_out, k_out); q_out may be q, k_out may be k.  inverse: turns back (not with norm
        weights)."""
        return _on(self.device, stream, self._call, q, k, pos, q_out, k_out, inverse)

    def _call(self, q, k, pos, q_out, k_out, inverse, s):
        if k is None and k_out is not None:
            raise ValueError("RotaryND: k_out without k")
        if pos.get_device() != self.device.index:
            raise ValueError(f"RotaryND: every tensor must be on {self.device}, got pos on {pos.device}")
        if q_out is None:
            q_out = torch.empty_like(q)
        if k_out is None and k is not None:
            k_out = torch.empty_like(k)
        lib.rope_nd(q, k, self.plan, pos, q_out, k_out, self.q_norm, None if k is None else self.k_norm, inverse,
                    self.eps, s)
        return q_out, k_out
