"""e4m3 weights and tokens with one scale per block of 128: the binding of include/qmm.h's qmm_f8_* calls.

    m = F8Matrix.quantize(w)           # w [M, K] or [E, M, K]: codes and scales of 128 x 128 blocks
    y = m.linear(x)                    # tokens quantized in the call, any number of them
    y = m.linear_id(x, ids)            # expert-indexed: ids [N, S]
    t = f8_quantize(x); y = m.gemm(t)  # one quantization for several matrices

Training (no autograd: results carry no gradient history whatever their inputs require, every gradient is a call):

    xq, xt = f8_quantize_pair(x)                  # along K, and along the tokens
    gq, gt = f8_quantize_pair(dy)
    dx = m.transposed().gemm(gq)
    dw = f8_wgrad(gt, xt)

Where a call takes `out`, that tensor's type is the output's.  As everywhere in this package the functions check tensor
metadata, allocate outputs and workspaces with torch and pass pointers; the current stream of the tensors' device is used,
whichever device is current.
"""

import ctypes

import torch

from ._lib import check, lib

BLOCK = 128
_DT = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_CODES = (torch.uint8, torch.float8_e4m3fn)


class _Seen(dict):
    """Sizes of calls seen before, which only the library computes: 1024 at most, then it starts anew."""

    def __setitem__(self, key, value):
        if len(self) >= 1024:
            self.clear()
        super().__setitem__(key, value)


def _padded(n):
    return (n + BLOCK - 1) // BLOCK * BLOCK


# torch's own shortcuts, which cost less host time, where it has them
_current_device = getattr(torch._C, "_cuda_getDevice", None) or (lambda: torch.cuda.current_device())
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _call(device, fn, *args):
    """fn(*args, the current stream of device), with device (an index) current; raises on an error status."""
    if _current_device() == device:
        status = fn(*args, _current_stream(device))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _current_stream(device))
    if status:
        check(status)


def _tensor(t, name, dtypes, dim=None):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}; expected one of {[str(d) for d in dtypes]}")
    if dim is not None and t.dim() not in dim:
        raise ValueError(f"{name} must be a tensor of {' or '.join(str(d) for d in dim)} dimensions")


def _shape(t, name, shape):
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}; expected {tuple(shape)}")


def _place(device, *named):
    """Every (tensor, name) is a contiguous tensor on device (an index; None: the first one's)."""
    for t, name in named:
        d = t.get_device()
        if d < 0:
            raise ValueError(f"{name} must be a device tensor")
        if device is None:
            device = d
        elif d != device:
            raise ValueError(f"{name} is on cuda:{d}; expected cuda:{device}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    return device


def _rows(x, name):
    """Row stride of a [N, K] device tensor whose rows are contiguous (a slice of wider rows is taken as it is)."""
    if not x.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    N, K = x.shape
    ld, step = x.stride()
    if N == 0 or K == 0:
        return K
    if K > 1 and step != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if N == 1:
        return K
    if ld < K:
        raise ValueError(f"{name} has overlapping rows")
    return ld


def _spans(codes, scales):
    """First byte and the byte behind the last of two contiguous tensors."""
    c, s = codes.data_ptr(), scales.data_ptr()
    return c, c + codes.numel() * codes.element_size(), s, s + scales.numel() * scales.element_size()


def _empty(shape, dtype, device):
    """torch.empty of two or three dimensions; with the strides named it takes 1.3 us, not 1.7."""
    n = shape[-1]
    strides = (n, 1) if len(shape) == 2 else (shape[1] * n, n, 1)
    return torch.empty_strided(shape, strides, dtype=dtype, device=_DEVICES[device])


def _out(out, shape, dtype, device, name="out"):
    if out is None:
        return _empty(shape, dtype, device)
    _tensor(out, name, _DT)
    _shape(out, name, shape)
    _place(device, (out, name))
    return out


_DEVICES = [torch.device("cuda", i) for i in range(64)]


def _dtype(t):
    if t not in _DT:
        raise ValueError(f"output dtype {t}; expected one of {[str(d) for d in _DT]}")
    return t


class F8Tokens:
    """Quantized rows: codes [R, padded C] uint8 and scales [padded C / 128, R] fp32.  C, the length of the quantized
    axis, is K for tokens ([N, K]) and the number of tokens for a transposed quantization (`channels` rows).  With a plan
    (f8_quantize_t) C is its pairs and a row has plan.routed codes, each expert's pairs padded on their own.  transposed:
    True and False as f8_quantize_t and f8_quantize made it, None for a caller's own codes, which may be either."""

    __slots__ = ("_codes", "_scales", "_buffer", "ptrs", "pitch", "rows", "length", "plan", "device", "transposed")

    def __init__(self, codes, scales, rows, length, plan=None):
        _tensor(codes, "codes", _CODES, (2,))
        _tensor(scales, "scales", (torch.float32,), (2,))
        # with a plan the native calls take the pitch from the plan's sizes
        pitch = plan.routed if plan is not None else _padded(length)
        if plan is not None and length != plan.N * plan.S:
            raise ValueError(f"{length} tokens; the plan has {plan.N} x {plan.S} pairs")
        _shape(codes, "codes", (rows, pitch))
        _shape(scales, "scales", (pitch // BLOCK, rows))
        self.device = _place(None, (codes, "codes"), (scales, "scales"))
        self._codes, self._scales, self._buffer = codes, scales, None
        self.ptrs = codes.data_ptr(), scales.data_ptr()
        self.pitch, self.rows, self.length, self.plan, self.transposed = pitch, rows, length, plan, None

    @classmethod
    def _empty(cls, rows, pitch, length, on, device, transposed, plan=None):
        """Room for codes and scales in one buffer; the tensors are made when asked for."""
        t = object.__new__(cls)
        t._buffer = torch.empty(rows * pitch + rows * (pitch // BLOCK) * 4, dtype=torch.uint8, device=on)
        t._codes = t._scales = None
        at = t._buffer.data_ptr()
        t.ptrs = at, at + rows * pitch
        t.pitch, t.rows, t.length, t.plan, t.device, t.transposed = pitch, rows, length, plan, device, transposed
        return t

    @property
    def codes(self):
        if self._codes is None:
            self._codes = self._buffer[:self.rows * self.pitch].view(self.rows, self.pitch)
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            self._scales = self._buffer[self.rows * self.pitch:].view(torch.float32).view(self.pitch // BLOCK, self.rows)
        return self._scales

    def values(self):
        """The values the codes stand for, [R, C] fp32 (in torch: for inspection, not a product path)."""
        v = self.codes.view(torch.float8_e4m3fn).float().unflatten(1, (-1, BLOCK)) * self.scales.t().unsqueeze(2)
        return v.flatten(1)[:, :self.length]


def _quantize(x, along_k, along_n):
    _tensor(x, "x", _DT, (2, 3))
    if x.shape[-1] == 0:
        raise ValueError("x has no columns")
    if x.dim() == 3:
        if not x.is_contiguous():
            raise ValueError("x of three dimensions must be contiguous")
        x = x.view(-1, x.shape[2])
    N, K = x.shape
    ld = K if x.is_contiguous() and x.is_cuda else _rows(x, "x")
    device, d = x.device, x.get_device()
    r = F8Tokens._empty(N, _padded(K), K, device, d, False) if along_k else None
    c = F8Tokens._empty(K, _padded(N), N, device, d, True) if along_n else None
    _call(d, lib.qmm_f8_quantize, x.data_ptr(), _DT[x.dtype], ld, N, K, *(r.ptrs if along_k else (None, None)),
          *(c.ptrs if along_n else (None, None)))
    return r, c


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
    _tensor(x, "x", _DT, (2, 3))
    per_slot = plan.per_slot_rows(x, "x")
    x2 = x.reshape(-1, x.shape[-1]) if x.dim() == 3 else x
    K = x2.shape[1]
    if K == 0:
        raise ValueError("x has no columns")
    ld = K if x2.is_contiguous() and x2.is_cuda else _rows(x2, "x")
    d = x.get_device()
    at = plan.place(d)
    t = F8Tokens._empty(K, plan.routed, plan.N * plan.S, x.device, d, True, plan)
    _call(d, lib.qmm_f8_quantize_routed, x2.data_ptr(), _DT[x.dtype], ld, plan.N, plan.S, per_slot, K, plan.n_experts,
          at, *t.ptrs)
    return t


_wgrad_need = _Seen()  # workspace bytes of the sizes seen


def f8_wgrad(g: F8Tokens, x: F8Tokens, plan=None, out: torch.Tensor = None, dtype=torch.float32) -> torch.Tensor:
    """dw [M, K] = g^T x (dw [E, M, K] with a plan), g and x quantized along the same tokens by f8_quantize_t."""
    if g.length != x.length or g.pitch != x.pitch:
        raise ValueError(f"g has {g.length} tokens, x has {x.length}")
    if g.plan is not plan or x.plan is not plan:
        raise ValueError("g and x must be quantized with the plan of this call (none without one)")
    if g.transposed is False or x.transposed is False:
        raise ValueError("g and x must be quantized along the tokens (f8_quantize_t)")
    M, K, device = g.rows, x.rows, g.device
    if x.device != device:
        raise ValueError(f"x is on cuda:{x.device}, g on cuda:{device}")
    shape = (M, K) if plan is None else (plan.n_experts, M, K)
    at = None if plan is None else plan.place(device)
    dw = _out(out, shape, _dtype(dtype), device)
    ptrs = g.ptrs + x.ptrs
    if plan is None:
        nb = _wgrad_need.get((g.length, M, K))
        if nb is None:
            nb = _wgrad_need[g.length, M, K] = lib.qmm_f8_wgrad_workspace_bytes(g.length, M, K)
        ws = torch.empty(nb, dtype=torch.uint8, device=_DEVICES[device]) if nb else None
        _call(device, lib.qmm_f8_wgrad, *ptrs, g.length, M, K, dw.data_ptr(), _DT[dw.dtype],
              ws.data_ptr() if nb else None, nb)
    else:
        _call(device, lib.qmm_f8_wgrad_id, *ptrs, plan.N, plan.S, M, K, plan.n_experts, at, dw.data_ptr(),
              _DT[dw.dtype])
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
        self._spans = _spans(codes, scales)
        self._need = _Seen()  # workspace bytes of the calls seen: N of linear, ~N of gemm, (N, S, per_slot) of linear_id
        h = ctypes.c_void_p()
        with torch.cuda.device(device):
            check(lib.qmm_f8_create(ctypes.byref(h), codes.data_ptr(), scales.data_ptr(), E, M, K))
        self._h = h

    @classmethod
    def _empty(cls, E, M, K, device, stacked):
        lead = (E,) if stacked else ()
        on = _DEVICES[device]
        codes = torch.empty(lead + (M, _padded(K)), dtype=torch.uint8, device=on)
        scales = torch.empty(lead + (_padded(M) // BLOCK, _padded(K) // BLOCK), dtype=torch.float32, device=on)
        return cls(codes, scales, M, K, E)

    @classmethod
    def quantize(cls, w: torch.Tensor) -> "F8Matrix":
        """w [M, K] or [E, M, K] (fp32, fp16 or bf16, contiguous)."""
        _tensor(w, "w", _DT, (2, 3))
        device = _place(None, (w, "w"))
        if w.numel() == 0:
            raise ValueError("w is empty")
        m = cls._empty(w.shape[0] if w.dim() == 3 else 1, w.shape[-2], w.shape[-1], device, w.dim() == 3)
        m.update(w)
        return m

    def close(self):
        h, self._h = getattr(self, "_h", None), None
        if h is not None and h.value is not None:
            p = ctypes.c_void_p(h.value)
            h.value = None  # whoever else has it sees that it is gone
            check(lib.qmm_f8_destroy(p))

    def __copy__(self):
        """Another handle of the same codes and scales."""
        return F8Matrix(self.codes, self.scales, self.M, self.K, self.n_experts)

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
        _tensor(w, "w", _DT, (2, 3))
        _shape(w, "w", ((self.n_experts,) if w.dim() == 3 or self.n_experts > 1 else ()) + (self.M, self.K))
        _place(self.device, (w, "w"))
        t = (None, None)
        if transposed is not None:
            self._check_transpose(transposed)
            t = transposed.codes.data_ptr(), transposed.scales.data_ptr()
        _call(self.device, lib.qmm_f8_quantize_weight, w.data_ptr(), _DT[w.dtype], self.n_experts, self.M, self.K,
              self.codes.data_ptr(), self.scales.data_ptr(), *t)

    def _check_transpose(self, m):
        if not isinstance(m, F8Matrix) or (m.M, m.K, m.n_experts) != (self.K, self.M, self.n_experts):
            raise ValueError(f"the transpose must be an F8Matrix of {self.n_experts} x [{self.K}, {self.M}]")
        (c0, c1, s0, s1), (tc0, tc1, ts0, ts1) = self._spans, m._spans
        if (c0 < tc1 and tc0 < c1) or (s0 < ts1 and ts0 < s1) or (c0 < ts1 and ts0 < c1) or (s0 < tc1 and tc0 < s1):
            raise ValueError("the transpose must have buffers of its own")
        if m.device != self.device:
            raise ValueError(f"the transpose is on cuda:{m.device}; the matrix is on cuda:{self.device}")

    def transposed(self, out: "F8Matrix" = None) -> "F8Matrix":
        """The matrix of W^T: the same codes and scales, transposed (into `out`'s buffers if given)."""
        if out is None:
            out = F8Matrix._empty(self.n_experts, self.K, self.M, self.device, self.codes.dim() == 3)
        self._check_transpose(out)
        _call(self.device, lib.qmm_f8_transpose, self._h, out.codes.data_ptr(), out.scales.data_ptr())
        return out

    def dequantize(self, expert: int = 0, dtype=torch.float32) -> torch.Tensor:
        out = _out(None, (self.M, self.K), _dtype(dtype), self.device)
        _call(self.device, lib.qmm_f8_dequantize, self._h, int(expert), out.data_ptr(), _DT[dtype])
        return out

    def linear(self, x: torch.Tensor, out_dtype=None, out: torch.Tensor = None) -> torch.Tensor:
        """x [N, K] (rows may be strided) -> y [N, M] of x's type (or out_dtype): quantization and product."""
        self._dense("linear")
        _tensor(x, "x", _DT, (2,))
        N, K = x.shape
        if K != self.K:
            raise ValueError(f"x has K={K}, matrix has K={self.K}")
        ld = K if x.is_contiguous() and x.is_cuda else _rows(x, "x")
        d = self.device
        if x.get_device() != d:
            raise ValueError(f"x is on {x.device}; the matrix is on cuda:{d}")
        if out is None:
            y = _empty((N, self.M), _dtype(out_dtype) if out_dtype else x.dtype, d)
        else:
            y = _out(out, (N, self.M), x.dtype, d)
        nb = self._need.get(N)
        if nb is None:
            nb = self._need[N] = lib.qmm_f8_linear_workspace_bytes(self._h, N)
        ws = torch.empty(nb, dtype=torch.uint8, device=_DEVICES[d]) if nb else None
        _call(d, lib.qmm_f8_linear, self._h, x.data_ptr(), _DT[x.dtype], ld, N, y.data_ptr(), _DT[y.dtype],
              ws.data_ptr() if nb else None, nb)
        return y

    def _tokens(self, t):
        if not isinstance(t, F8Tokens) or t.plan is not None:
            raise ValueError("tokens must come from f8_quantize")
        if t.length != self.K:
            raise ValueError(f"tokens have K={t.length}, matrix has K={self.K}")
        if t.transposed:
            raise ValueError("tokens are quantized along the tokens (f8_quantize_t); a product takes them along K (f8_quantize)")
        if t.device != self.device:
            raise ValueError(f"tokens are on cuda:{t.device}; the matrix is on cuda:{self.device}")

    def gemm(self, tokens: F8Tokens, out_dtype=torch.float32, out: torch.Tensor = None) -> torch.Tensor:
        """Quantized tokens [N, K] -> y [N, M]."""
        self._dense("gemm")
        self._tokens(tokens)
        N = tokens.rows
        y = _out(out, (N, self.M), _dtype(out_dtype), self.device)
        nb = self._need.get(~N)
        if nb is None:
            nb = self._need[~N] = lib.qmm_f8_gemm_workspace_bytes(self._h, N)
        ws = torch.empty(nb, dtype=torch.uint8, device=_DEVICES[self.device]) if nb else None
        _call(self.device, lib.qmm_f8_gemm, self._h, *tokens.ptrs, N, y.data_ptr(),
              _DT[y.dtype], ws.data_ptr() if nb else None, nb)
        return y

    def linear_id(self, x: torch.Tensor, ids: torch.Tensor, out_dtype=None, out: torch.Tensor = None) -> torch.Tensor:
        """ids [N, S] int32 (-1: an empty slot); x [N, S, K] (one row per slot) or [N, K], contiguous -> y [N, S, M]."""
        _tensor(x, "x", _DT, (2, 3))
        _tensor(ids, "ids", (torch.int32,), (2,))
        N, S = ids.shape
        if S < 1:
            raise ValueError("ids has no slots")
        per_slot = int(x.dim() == 3)
        _shape(x, "x", (N, S, self.K) if per_slot else (N, self.K))
        _place(self.device, (x, "x"), (ids, "ids"))
        y = _out(out, (N, S, self.M), _dtype(out_dtype or x.dtype), self.device)
        nb = self._need.get((N, S, per_slot))
        if nb is None:
            nb = self._need[N, S, per_slot] = lib.qmm_f8_linear_id_workspace_bytes(self._h, N, S, per_slot)
        ws = torch.empty(nb, dtype=torch.uint8, device=x.device) if nb else None
        _call(self.device, lib.qmm_f8_linear_id, self._h, x.data_ptr(), _DT[x.dtype], N, S, per_slot, ids.data_ptr(),
              y.data_ptr(), _DT[y.dtype], ws.data_ptr() if nb else None, nb)
        return y

    def gemm_id(self, tokens: F8Tokens, plan, out_dtype=torch.float32, out: torch.Tensor = None) -> torch.Tensor:
        """Quantized tokens (N rows, shared by a token's slots, or N * S) and the plan of ids [N, S] -> y [N, S, M]."""
        if plan.n_experts != self.n_experts:
            raise ValueError(f"the plan has {plan.n_experts} experts, the matrix {self.n_experts}")
        per_slot = plan.per_slot(tokens.rows, "tokens")
        self._tokens(tokens)
        at = plan.place(self.device)
        y = _out(out, (plan.N, plan.S, self.M), _dtype(out_dtype), self.device)
        _call(self.device, lib.qmm_f8_gemm_id, self._h, *tokens.ptrs, plan.N, plan.S,
              per_slot, at, y.data_ptr(), _DT[y.dtype])
        return y
