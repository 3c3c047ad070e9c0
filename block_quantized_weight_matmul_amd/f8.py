"""e4m3 weights and tokens with one scale per block of 128: the binding of include/qmm.h's qmm_f8_* calls.

    m = F8Matrix.quantize(w)           # w [M, K] or [E, M, K]: codes and scales of 128 x 128 blocks
    y = m.linear(x)                    # tokens quantized in the call, any number of them
    y = m.linear_id(x, ids)            # expert-indexed: ids [N, S]
    t = f8_quantize(x); y = m.gemm(t)  # one quantization for several matrices

Training (no autograd: every gradient is a call):

    xq, xt = f8_quantize_pair(x)                  # along K, and along the tokens
    gq, gt = f8_quantize_pair(dy)
    dx = m.transposed().gemm(gq)
    dw = f8_wgrad(gt, xt)

As everywhere in this package the functions check tensor metadata, allocate outputs and workspaces with torch and
pass pointers; the current stream of the tensors' device is used, whichever device is current.
"""

import ctypes

import torch

from ._lib import check, lib

BLOCK = 128
_DT = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_CODES = (torch.uint8, torch.float8_e4m3fn)


def _padded(n):
    return (n + BLOCK - 1) // BLOCK * BLOCK


class _Device:
    """The tensors' device made current for a library call, and its current stream."""

    __slots__ = ("index", "back")

    def __init__(self, device):
        self.index, self.back = device.index, None

    def __enter__(self):
        now = torch.cuda.current_device()
        if now != self.index:
            torch.cuda.set_device(self.index)
            self.back = now
        return torch.cuda.current_stream(self.index).cuda_stream

    def __exit__(self, *_):
        if self.back is not None:
            torch.cuda.set_device(self.back)


def _tensor(t, name, dtypes, dim=None):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}; expected one of {[str(d) for d in dtypes]}")
    if dim is not None and t.dim() not in dim:
        raise ValueError(f"{name} must be a tensor of {' or '.join(str(d) for d in dim)} dimensions")


def _shape(t, name, shape):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}; expected {tuple(shape)}")


def _place(device, *named):
    """Every (tensor, name) is a contiguous tensor on `device` (None: the first one's)."""
    for t, name in named:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a device tensor")
        if device is None:
            device = t.device
        elif t.device != device:
            raise ValueError(f"{name} is on {t.device}; expected {device}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    return device


def _rows(x, name):
    """Row stride of a [N, K] device tensor whose rows are contiguous (a slice of wider rows is taken as it is)."""
    if not x.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    N, K = x.shape
    if N == 0 or K == 0:
        return K
    if K > 1 and x.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if N == 1:
        return K
    if x.stride(0) < K:
        raise ValueError(f"{name} has overlapping rows")
    return x.stride(0)


def _out(out, shape, dtype, device, name="out"):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _tensor(out, name, tuple(_DT))
    _shape(out, name, shape)
    _place(device, (out, name))
    return out


def _dtype(t):
    if t not in _DT:
        raise ValueError(f"output dtype {t}; expected one of {[str(d) for d in _DT]}")
    return t


class F8Tokens:
    """Quantized rows: codes [R, padded C] uint8 and scales [padded C / 128, R] fp32.  C, the length of the quantized
    axis, is K for tokens ([N, K]) and the number of tokens for a transposed quantization (`channels` rows)."""

    __slots__ = ("codes", "scales", "rows", "length", "plan")

    def __init__(self, codes, scales, rows, length, plan=None):
        _tensor(codes, "codes", _CODES, (2,))
        _tensor(scales, "scales", (torch.float32,), (2,))
        pitch = codes.shape[1] if plan is not None else _padded(length)
        _shape(codes, "codes", (rows, pitch))
        _shape(scales, "scales", (pitch // BLOCK, rows))
        _place(None, (codes, "codes"), (scales, "scales"))
        self.codes, self.scales, self.rows, self.length, self.plan = codes, scales, rows, length, plan

    def values(self):
        """The values the codes stand for, [R, C] fp32 (in torch: for inspection, not a product path)."""
        v = self.codes.view(torch.float8_e4m3fn).float().unflatten(1, (-1, BLOCK)) * self.scales.t().unsqueeze(2)
        return v.flatten(1)[:, :self.length]


def _empty_tokens(rows, pitch, device):
    return (torch.empty((rows, pitch), dtype=torch.uint8, device=device),
            torch.empty((pitch // BLOCK, rows), dtype=torch.float32, device=device))


def _quantize(x, along_k, along_n):
    _tensor(x, "x", tuple(_DT), (2, 3))
    if x.dim() == 3:
        if not x.is_contiguous():
            raise ValueError("x of three dimensions must be contiguous")
        x = x.view(-1, x.shape[2])
    N, K = x.shape
    if K == 0:
        raise ValueError("x has no columns")
    ld = _rows(x, "x")
    r = _empty_tokens(N, _padded(K), x.device) if along_k else (None, None)
    c = _empty_tokens(K, _padded(N), x.device) if along_n else (None, None)
    p = [t.data_ptr() if t is not None else None for t in (*r, *c)]
    with _Device(x.device) as stream:
        check(lib.qmm_f8_quantize(x.data_ptr(), _DT[x.dtype], ld, N, K, *p, stream))
    return (F8Tokens(*r, N, K) if along_k else None), (F8Tokens(*c, K, N) if along_n else None)


def f8_quantize(x: torch.Tensor) -> F8Tokens:
    """x [N, K] (fp32, fp16 or bf16; rows may be strided) or [N, S, K] quantized as tokens: one scale per 128 values
    along K."""
    return _quantize(x, True, False)[0]


def f8_quantize_pair(x: torch.Tensor):
    """(f8_quantize(x), f8_quantize_t(x)) in one pass over x."""
    return _quantize(x, True, True)


def f8_quantize_t(x: torch.Tensor, plan=None) -> F8Tokens:
    """x [N, K] quantized along the tokens, K rows of codes: the operands of f8_wgrad.  With a plan (of ids [N, S]) the
    rows are the plan's pairs, expert by expert: x [N, K] (shared by a token's slots) or [N, S, K] / [N * S, K]."""
    if plan is None:
        return _quantize(x, False, True)[1]
    _tensor(x, "x", tuple(_DT), (2, 3))
    per_slot = plan.per_slot_rows(x, "x")
    x2 = x.reshape(-1, x.shape[-1]) if x.dim() == 3 else x
    K = x2.shape[1]
    if K == 0:
        raise ValueError("x has no columns")
    ld = _rows(x2, "x")
    _place(x.device, (plan.data, "plan"))
    codes, scales = _empty_tokens(K, lib.qmm_f8_routed_tokens(plan.N * plan.S, plan.n_experts), x.device)
    with _Device(x.device) as stream:
        check(lib.qmm_f8_quantize_routed(x2.data_ptr(), _DT[x.dtype], ld, plan.N, plan.S, per_slot, K, plan.n_experts,
                                         plan.data.data_ptr(), codes.data_ptr(), scales.data_ptr(), stream))
    return F8Tokens(codes, scales, K, plan.N * plan.S, plan)


def f8_wgrad(g: F8Tokens, x: F8Tokens, plan=None, out: torch.Tensor = None, dtype=torch.float32) -> torch.Tensor:
    """dw [M, K] = g^T x (dw [E, M, K] with a plan), g and x quantized along the same tokens by f8_quantize_t."""
    if g.length != x.length or g.codes.shape[1] != x.codes.shape[1]:
        raise ValueError(f"g has {g.length} tokens, x has {x.length}")
    if g.plan is not plan or x.plan is not plan:
        raise ValueError("g and x must be quantized with the plan of this call (none without one)")
    M, K = g.rows, x.rows
    device = _place(None, (g.codes, "g"), (x.codes, "x"))
    shape = (M, K) if plan is None else (plan.n_experts, M, K)
    dw = _out(out, shape, _dtype(dtype), device)
    ptrs = g.codes.data_ptr(), g.scales.data_ptr(), x.codes.data_ptr(), x.scales.data_ptr()
    with _Device(device) as stream:
        if plan is None:
            check(lib.qmm_f8_wgrad(*ptrs, g.length, M, K, dw.data_ptr(), _DT[dw.dtype], stream))
        else:
            _place(device, (plan.data, "plan"))
            check(lib.qmm_f8_wgrad_id(*ptrs, plan.N, plan.S, M, K, plan.n_experts, plan.data.data_ptr(), dw.data_ptr(),
                                      _DT[dw.dtype], stream))
    return dw


class F8Matrix:
    """e4m3 weights on the device: one matrix [M, K] or E stacked experts [E, M, K].

    codes  [M, padded K] or [E, M, padded K], uint8 or float8_e4m3fn, zero past K (padded: next multiple of 128).
    scales [padded M / 128, padded K / 128] or with E in front, fp32.
    Both are borrowed (kept referenced here) for the life of the object; `update` rewrites them in stream order."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, M: int, K: int, n_experts: int = 1):
        self._h = None
        M, K, E = int(M), int(K), int(n_experts)
        if min(M, K, E) < 1:
            raise ValueError("M, K and n_experts must be positive")
        _tensor(codes, "codes", _CODES)
        _tensor(scales, "scales", (torch.float32,))
        Kp, R, G = _padded(K), _padded(M) // BLOCK, _padded(K) // BLOCK
        stacked = codes.dim() == 3
        if E > 1 and not stacked:
            raise ValueError("codes of stacked experts must have 3 dimensions")
        lead = (E,) if stacked else ()
        _shape(codes, "codes", lead + (M, Kp))
        _shape(scales, "scales", ((E,) if scales.dim() == 3 or E > 1 else ()) + (R, G))
        device = _place(None, (codes, "codes"), (scales, "scales"))
        self.M, self.K, self.n_experts, self.codes, self.scales, self.device = M, K, E, codes, scales, device
        h = ctypes.c_void_p()
        with _Device(device):
            check(lib.qmm_f8_create(ctypes.byref(h), codes.data_ptr(), scales.data_ptr(), E, M, K))
        self._h = h

    @classmethod
    def _empty(cls, E, M, K, device, stacked):
        lead = (E,) if stacked else ()
        codes = torch.empty(lead + (M, _padded(K)), dtype=torch.uint8, device=device)
        scales = torch.empty(lead + (_padded(M) // BLOCK, _padded(K) // BLOCK), dtype=torch.float32, device=device)
        return cls(codes, scales, M, K, E)

    @classmethod
    def quantize(cls, w: torch.Tensor) -> "F8Matrix":
        """w [M, K] or [E, M, K] (fp32, fp16 or bf16, contiguous)."""
        _tensor(w, "w", tuple(_DT), (2, 3))
        device = _place(None, (w, "w"))
        if w.numel() == 0:
            raise ValueError("w is empty")
        m = cls._empty(w.shape[0] if w.dim() == 3 else 1, w.shape[-2], w.shape[-1], device, w.dim() == 3)
        m.update(w)
        return m

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value is not None:
            check(lib.qmm_f8_destroy(self._h))
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self):
        return self._h

    def _dense(self, what):
        if self.n_experts != 1:
            raise ValueError(f"{what} needs a single matrix; this one stacks {self.n_experts} experts")

    def update(self, w: torch.Tensor, transposed: "F8Matrix" = None) -> None:
        """Quantize new weights into this matrix' buffers (and their transpose into `transposed`'s, from the same pass)."""
        _tensor(w, "w", tuple(_DT), (2, 3))
        _shape(w, "w", ((self.n_experts,) if w.dim() == 3 or self.n_experts > 1 else ()) + (self.M, self.K))
        _place(self.device, (w, "w"))
        t = (None, None)
        if transposed is not None:
            self._check_transpose(transposed)
            t = transposed.codes.data_ptr(), transposed.scales.data_ptr()
        with _Device(self.device) as stream:
            check(lib.qmm_f8_quantize_weight(w.data_ptr(), _DT[w.dtype], self.n_experts, self.M, self.K,
                                             self.codes.data_ptr(), self.scales.data_ptr(), *t, stream))

    def _check_transpose(self, m):
        if not isinstance(m, F8Matrix) or (m.M, m.K, m.n_experts) != (self.K, self.M, self.n_experts):
            raise ValueError(f"the transpose must be an F8Matrix of {self.n_experts} x [{self.K}, {self.M}]")
        if m is self or m.codes.data_ptr() == self.codes.data_ptr():
            raise ValueError("the transpose must have buffers of its own")
        _place(self.device, (m.codes, "the transpose's codes"))

    def transposed(self, out: "F8Matrix" = None) -> "F8Matrix":
        """The matrix of W^T: the same codes and scales, transposed (into `out`'s buffers if given)."""
        if out is None:
            out = F8Matrix._empty(self.n_experts, self.K, self.M, self.device, self.codes.dim() == 3)
        self._check_transpose(out)
        with _Device(self.device) as stream:
            check(lib.qmm_f8_transpose(self._h, out.codes.data_ptr(), out.scales.data_ptr(), stream))
        return out

    def dequantize(self, expert: int = 0, dtype=torch.float32) -> torch.Tensor:
        out = torch.empty((self.M, self.K), dtype=_dtype(dtype), device=self.device)
        with _Device(self.device) as stream:
            check(lib.qmm_f8_dequantize(self._h, int(expert), out.data_ptr(), _DT[dtype], stream))
        return out

    def linear(self, x: torch.Tensor, out_dtype=None, out: torch.Tensor = None) -> torch.Tensor:
        """x [N, K] (rows may be strided) -> y [N, M] of x's type (or out_dtype): quantization and product."""
        self._dense("linear")
        _tensor(x, "x", tuple(_DT), (2,))
        N = x.shape[0]
        if x.shape[1] != self.K:
            raise ValueError(f"x has K={x.shape[1]}, matrix has K={self.K}")
        if x.device != self.device:
            raise ValueError(f"x is on {x.device}; the matrix is on {self.device}")
        ld = _rows(x, "x")
        y = _out(out, (N, self.M), _dtype(out_dtype or x.dtype), self.device)
        nb = lib.qmm_f8_linear_workspace_bytes(self._h, N)
        ws = torch.empty(nb, dtype=torch.uint8, device=self.device) if nb else None
        with _Device(self.device) as stream:
            check(lib.qmm_f8_linear(self._h, x.data_ptr(), _DT[x.dtype], ld, N, y.data_ptr(), _DT[y.dtype],
                                    ws.data_ptr() if nb else None, nb, stream))
        return y

    def _tokens(self, t, rows):
        if not isinstance(t, F8Tokens) or t.plan is not None:
            raise ValueError("tokens must come from f8_quantize")
        if t.length != self.K:
            raise ValueError(f"tokens have K={t.length}, matrix has K={self.K}")
        if rows is not None and t.rows != rows:
            raise ValueError(f"{t.rows} rows of tokens; expected {rows}")
        _place(self.device, (t.codes, "tokens"))

    def gemm(self, tokens: F8Tokens, out_dtype=torch.float32, out: torch.Tensor = None) -> torch.Tensor:
        """Quantized tokens [N, K] -> y [N, M]."""
        self._dense("gemm")
        self._tokens(tokens, None)
        N = tokens.rows
        y = _out(out, (N, self.M), _dtype(out_dtype), self.device)
        nb = lib.qmm_f8_gemm_workspace_bytes(self._h, N)
        ws = torch.empty(nb, dtype=torch.uint8, device=self.device) if nb else None
        with _Device(self.device) as stream:
            check(lib.qmm_f8_gemm(self._h, tokens.codes.data_ptr(), tokens.scales.data_ptr(), N, y.data_ptr(),
                                  _DT[y.dtype], ws.data_ptr() if nb else None, nb, stream))
        return y

    def linear_id(self, x: torch.Tensor, ids: torch.Tensor, out_dtype=None, out: torch.Tensor = None) -> torch.Tensor:
        """ids [N, S] int32 (-1: an empty slot); x [N, S, K] (one row per slot) or [N, K], contiguous -> y [N, S, M]."""
        _tensor(x, "x", tuple(_DT), (2, 3))
        _tensor(ids, "ids", (torch.int32,), (2,))
        N, S = ids.shape
        if S < 1:
            raise ValueError("ids has no slots")
        per_slot = int(x.dim() == 3)
        _shape(x, "x", (N, S, self.K) if per_slot else (N, self.K))
        _place(self.device, (x, "x"), (ids, "ids"))
        y = _out(out, (N, S, self.M), _dtype(out_dtype or x.dtype), self.device)
        nb = lib.qmm_f8_linear_id_workspace_bytes(self._h, N, S, per_slot)
        ws = torch.empty(nb, dtype=torch.uint8, device=self.device) if nb else None
        with _Device(self.device) as stream:
            check(lib.qmm_f8_linear_id(self._h, x.data_ptr(), _DT[x.dtype], N, S, per_slot, ids.data_ptr(), y.data_ptr(),
                                       _DT[y.dtype], ws.data_ptr() if nb else None, nb, stream))
        return y

    def gemm_id(self, tokens: F8Tokens, plan, out_dtype=torch.float32, out: torch.Tensor = None) -> torch.Tensor:
        """Quantized tokens (N rows, shared by a token's slots, or N * S) and the plan of ids [N, S] -> y [N, S, M]."""
        if plan.n_experts != self.n_experts:
            raise ValueError(f"the plan has {plan.n_experts} experts, the matrix {self.n_experts}")
        per_slot = plan.per_slot(tokens.rows, "tokens")
        self._tokens(tokens, None)
        _place(self.device, (plan.data, "plan"))
        y = _out(out, (plan.N, plan.S, self.M), _dtype(out_dtype), self.device)
        with _Device(self.device) as stream:
            check(lib.qmm_f8_gemm_id(self._h, tokens.codes.data_ptr(), tokens.scales.data_ptr(), plan.N, plan.S, per_slot,
                                     plan.data.data_ptr(), y.data_ptr(), _DT[y.dtype], stream))
        return y
