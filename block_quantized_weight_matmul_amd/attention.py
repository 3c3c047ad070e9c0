"""What a decoder layer does between its projections: the binding of include/qmm.h's qmm_head*, qmm_cache* and qmm_attend*
calls.

    cache = KVCache.empty(pages, 64, H, D, torch.bfloat16)        # or "e4m3"
    q, k = head_norm_rope(q, k, positions, inv_freq, q_weight, k_weight)
    out = attend_prompt(q, k, v, starts)                          # packed prompts, causal
    cache.write(k, v, slots)

and a decode step, one token of each sequence:

    q = cache.norm_rope_write(q, k, v, slots, positions, inv_freq, q_weight, k_weight)
    out = cache.attend(q, table, lengths)

A prompt that arrives in parts is written part by part; cache.read gives the whole sequences back for
attend_prompt(q, k, v, starts, k_starts).  Serving: there is no autograd and no gradient of these calls.

Queries, keys and values are [T, heads, D], slices of a wider buffer as they are (the last axis is contiguous).  As
everywhere in this package the functions check tensor metadata, allocate outputs and workspaces with torch and pass
pointers; the current stream of the tensors' device is used, whichever device is current.
"""

import ctypes
import struct

import torch

from ._lib import check, lib
from .f8 import _DT, _call, _current_device, _current_stream, _empty, _out, _place, _shape, _tensor

try:
    from . import _calls  # csrc/calls.cpp
except ImportError:  # not built, or for another torch or Python, which it tells: the same calls, through ctypes
    _calls = None

_HALF = {torch.float16: 1, torch.bfloat16: 2}
_CACHE = {torch.float16: 1, torch.bfloat16: 2, torch.uint8: 3, torch.float8_e4m3fn: 3}
_INT = torch.int32
_F32 = (torch.float32,)

# the argument structs of include/qmm.h
_pack_heads = struct.Struct("21q4if4x").pack
_pack_write = struct.Struct("8qi4x").pack
_pack_read = struct.Struct("7qi4x").pack
_pack_attend = struct.Struct("12qif").pack
_pack_prompt = struct.Struct("18q2if4x").pack


# --- argument checks ---------------------------------------------------------------------------
# _calls makes the checks of a call that is as it should be, and the call; a decode step's takes a few microseconds on the
# device, and here as long.  What it declines comes here, to be told what is wrong, or to be made: a tensor of a subclass,
# one on another device than the current one, an `out`.

def _here(x):
    """The current device, where native calls are made, if the tensor x lies there, else -1."""
    try:
        d = x.get_device()
    except AttributeError:
        return -1
    return d if _calls is not None and d >= 0 and d == _current_device() else -1


def _heads(x, name, dtypes, device=None):
    """(device, T, heads, D, stride of a token, stride of a head) of a [T, heads, D] device tensor."""
    _tensor(x, name, dtypes, (3,))
    d = x.get_device()
    if d < 0:
        raise ValueError(f"{name} must be a device tensor")
    if device is not None and d != device:
        raise ValueError(f"{name} is on cuda:{d}; expected cuda:{device}")
    if x.stride(2) != 1 and x.shape[2] > 1:
        raise ValueError(f"{name} must have a contiguous last axis")
    return (d, *x.shape, *x.stride()[:2])


def _vector(t, name, dtype, length, device):
    """Pointer of a contiguous vector of `length` elements on device."""
    _tensor(t, name, (dtype,), (1,))
    if t.shape[0] != length:
        raise ValueError(f"{name} has {t.shape[0]} elements; expected {length}")
    _place(device, (t, name))
    return t.data_ptr()


def _rotation(positions, inv_freq, T, device):
    """Pointers of the positions and frequencies, columns rotated."""
    if inv_freq is None:
        return 0, 0, 0
    if positions is None:
        raise ValueError("inv_freq needs positions")
    _tensor(inv_freq, "inv_freq", _F32, (1,))
    n = inv_freq.shape[0]
    return _vector(positions, "positions", _INT, T, device), _vector(inv_freq, "inv_freq", torch.float32, n, device), 2 * n


def _weights(q_weight, k_weight, D, device):
    """Pointers of the weights, their type."""
    if q_weight is None and k_weight is None:
        return 0, 0, 0
    dtype = k_weight.dtype if q_weight is None else getattr(q_weight, "dtype", None)
    if dtype not in _DT:
        _tensor(k_weight if q_weight is None else q_weight, "k_weight" if q_weight is None else "q_weight", _DT)
    return (0 if q_weight is None else _vector(q_weight, "q_weight", dtype, D, device),
            0 if k_weight is None else _vector(k_weight, "k_weight", dtype, D, device), _DT[dtype])


def _single(v):
    """A number as fp32 holds it; one beyond its range is infinite, which the library refuses."""
    return ctypes.c_float(v).value


def _result_type(dtype):
    if dtype not in _DT:
        raise ValueError(f"dtype {dtype}; expected one of {[str(d) for d in _DT]}")


def head_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, dtype=None):
    """(q', k'): every head of q [T, Hq, D] and k [T, H, D] divided by its root mean square and multiplied by its weight [D]
    (None: no norm), then its first 2 len(inv_freq) columns rotated by positions [T] (int32) times inv_freq (fp32; None: no
    rotation), column i with column i + len(inv_freq), or 2 i with 2 i + 1 where interleaved.  dtype: of the results."""
    d = _here(q)
    if d >= 0:
        made = _calls.head_norm_rope(d, _current_stream(d), q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, dtype)
        if made is not None:
            return made
    d, T, Hq, D, qt, qh = _heads(q, "q", _DT)
    xt = q.dtype
    _, Tk, H, Dk, kt, kh = _heads(k, "k", (xt,), d)
    if Tk != T or Dk != D:
        raise ValueError(f"k has shape {tuple(k.shape)}; q has {tuple(q.shape)}")
    if dtype is None:
        dtype = xt
    else:
        _result_type(dtype)
    pos, freq, R = _rotation(positions, inv_freq, T, d)
    qw, kw, wt = _weights(q_weight, k_weight, D, d)
    qo, ko = _empty((T, Hq, D), dtype, d), _empty((T, H, D), dtype, d)
    _call(d, lib.qmm_head_norm_rope, _pack_heads(
        q.data_ptr(), k.data_ptr(), 0, qw, kw, pos, freq, 0, qo.data_ptr(), ko.data_ptr(), qt, qh, kt, kh, 0, 0, T, Hq, H, D, R,
        _DT[xt], wt, _DT[dtype], 1 if interleaved else 0, _single(eps)))
    return qo, ko


class KVCache:
    """A paged cache of keys and values, k and v [pages, heads, page, D]: fp16, bf16, or e4m3 codes (uint8 or float8_e4m3fn)
    with fp32 scales [pages, heads, page], one per token and head.  page is a power of two from 16 on, D a multiple of 16 up
    to 256.  The tensors are kept referenced and written in place.

    A token's slot is its page times `page` plus its row there; a table int32 [B, W] names the pages of B sequences in
    order, entries past a sequence's last page may hold anything: no result depends on them."""

    def __init__(self, k, v, k_scales=None, v_scales=None):
        _tensor(k, "k", _CACHE, (4,))
        _tensor(v, "v", (k.dtype,), (4,))
        _shape(v, "v", k.shape)
        self.pages, self.heads, self.page, self.D = k.shape
        named = [(k, "k"), (v, "v")]
        if _CACHE[k.dtype] == 3:
            for s, name in ((k_scales, "k_scales"), (v_scales, "v_scales")):
                _tensor(s, name, _F32, (3,))
                _shape(s, name, k.shape[:3])
                named.append((s, name))
        elif k_scales is not None or v_scales is not None:
            raise ValueError("only an e4m3 cache has scales")
        self.device = _place(None, *named)
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.dtype = k.dtype if k.dtype in _HALF else torch.float8_e4m3fn
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            check(lib.qmm_cache_create(ctypes.byref(h), *(t.data_ptr() for t, _ in named), *([None] * (4 - len(named))),
                                       _CACHE[k.dtype], self.pages, self.page, self.heads, self.D))
        self._h = h
        # what the native calls take of it
        self._id = h.value, self.heads, self.D
        self._type = _CACHE[k.dtype]

    @classmethod
    def empty(cls, pages, page, heads, D, dtype=torch.bfloat16, device="cuda"):
        """A cache of zeros.  dtype: torch.float16, torch.bfloat16, torch.float8_e4m3fn or "e4m3"."""
        codes = dtype in ("e4m3", torch.float8_e4m3fn)
        if not codes and dtype not in _HALF:
            raise ValueError(f"cache dtype {dtype}; expected float16, bfloat16 or e4m3")
        shape = (pages, heads, page, D)
        made = [torch.zeros(shape, dtype=torch.uint8 if codes else dtype, device=device) for _ in "kv"]
        if codes:
            made += [torch.zeros(shape[:3], dtype=torch.float32, device=device) for _ in "kv"]
        return cls(*made)

    def close(self):
        h, self._h = getattr(self, "_h", None), None
        self._id = 0, 0, 0
        if h is not None and h.value is not None:
            lib.qmm_cache_destroy(h)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __copy__(self):
        return KVCache(self.k, self.v, self.k_scales, self.v_scales)

    def __deepcopy__(self, memo):
        return KVCache(*(None if t is None else t.clone() for t in (self.k, self.v, self.k_scales, self.v_scales)))

    def __reduce__(self):
        return KVCache, (self.k, self.v, self.k_scales, self.v_scales)

    def _kv(self, k, v):
        """Type, tokens and strides of keys and values."""
        _, T, H, D, kt, kh = _heads(k, "k", _DT, self.device)
        _, Tv, Hv, Dv, vt, vh = _heads(v, "v", (k.dtype,), self.device)
        if H != self.heads or D != self.D:
            raise ValueError(f"k has {H} heads of {D}; the cache has {self.heads} of {self.D}")
        if Tv != T or Hv != H or Dv != D:
            raise ValueError(f"v has shape {tuple(v.shape)}; k has {tuple(k.shape)}")
        return k.dtype, T, kt, kh, vt, vh

    def write(self, k, v, slots):
        """k and v [T, heads, D] to slots [T] (int32; negative ones and those past the last page are left out).  The slots
        of a call are distinct."""
        d = self.device
        if _here(k) == d and _calls.write(d, _current_stream(d), *self._id, k, v, slots):
            return
        xt, T, kt, kh, vt, vh = self._kv(k, v)
        at = _vector(slots, "slots", _INT, T, self.device)
        _call(self.device, lib.qmm_cache_write, self._h, _pack_write(k.data_ptr(), v.data_ptr(), at, kt, kh, vt, vh, T, _DT[xt]))

    def norm_rope_write(self, q, k, v, slots, positions, inv_freq, q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                        dtype=None):
        """head_norm_rope of q and k, then write of the keys and of v, in one launch and with the same bits; returns q'.
        dtype: of q' and, before they are quantized, of the keys; the cache's own unless that is e4m3 (then q's)."""
        d = self.device
        if _here(q) == d:
            made = _calls.norm_rope_write(d, _current_stream(d), *self._id, self._type, q, k, v, slots, positions, inv_freq, q_weight,
                                          k_weight, eps, interleaved, dtype)
            if made is not None:
                return made
        _, T, Hq, D, qt, qh = _heads(q, "q", _DT, d)
        xt, Tk, kt, kh, vt, vh = self._kv(k, v)
        if xt != q.dtype:
            raise ValueError(f"k has dtype {xt}; q has {q.dtype}")
        if Tk != T or D != self.D:
            raise ValueError(f"q has shape {tuple(q.shape)}; k has {tuple(k.shape)}")
        if dtype is None:
            dtype = self.dtype if self.dtype in _HALF else xt
        else:
            _result_type(dtype)
            if self.dtype in _HALF and dtype != self.dtype:
                raise ValueError(f"dtype {dtype}; the cache has {self.dtype}")
        pos, freq, R = _rotation(positions, inv_freq, T, d)
        qw, kw, wt = _weights(q_weight, k_weight, D, d)
        at = _vector(slots, "slots", _INT, T, d)
        o = _empty((T, Hq, D), dtype, d)
        _call(d, lib.qmm_cache_norm_rope_write, self._h, _pack_heads(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), qw, kw, pos, freq, at, o.data_ptr(), 0, qt, qh, kt, kh, vt, vh, T, Hq,
            self.heads, D, R, _DT[xt], wt, _DT[dtype], 1 if interleaved else 0, _single(eps)))
        return o

    def _table(self, table, B):
        _tensor(table, "table", (_INT,), (2,))
        if table.shape[0] != B:
            raise ValueError(f"table has {table.shape[0]} rows; expected {B}")
        _place(self.device, (table, "table"))
        return table.data_ptr(), table.shape[1]

    def read(self, table, starts, total, dtype=None, out=None):
        """(k, v) [total, heads, D]: sequence b's tokens as rows starts[b] .. starts[b + 1] - 1 (starts int32 [B + 1], not
        decreasing).  Rows of no sequence are not written: they stay as they were in `out`, a pair of tensors."""
        d = self.device
        if out is None and _here(table) == d:
            made = _calls.read(d, _current_stream(d), *self._id, self._type, table, starts, total, dtype)
            if made is not None:
                return made
        _tensor(starts, "starts", (_INT,), (1,))
        B = starts.shape[0] - 1
        if B < 0:
            raise ValueError("starts is empty")
        at, W = self._table(table, B)
        first = _vector(starts, "starts", _INT, B + 1, d)
        total = int(total)
        if total < 0:
            raise ValueError(f"total={total} is negative")
        shape = (total, self.heads, self.D)
        if out is None:
            dtype = (self.dtype if self.dtype in _HALF else torch.bfloat16) if dtype is None else dtype
            _result_type(dtype)
            k, v = _empty(shape, dtype, d), _empty(shape, dtype, d)
        else:
            k, v = out
            _out(k, shape, None, d, "out[0]")
            _out(v, shape, None, d, "out[1]")
            if v.dtype != k.dtype or dtype not in (None, k.dtype):
                raise ValueError("out must be two tensors of one dtype, that of the call")
            dtype = k.dtype
        _call(d, lib.qmm_cache_read, self._h, _pack_read(at, first, k.data_ptr(), v.data_ptr(), B, W, total, _DT[dtype]))
        return k, v

    def attend(self, q, table, lengths, scale=None, max_length=None, out=None):
        """Attention of one token per sequence, q [B, Hq, D] (fp16 or bf16, a 16-bit cache's own type), over the first
        lengths[b] (int32) tokens of each sequence; Hq a multiple of the cache's heads.  scale: of the scores, 1 / sqrt(D) by
        default.  max_length: the longest length where the host knows it, else the table's reach; it decides how the work
        is divided and nothing else."""
        d = self.device
        if out is None and _here(q) == d:
            made = _calls.attend(d, _current_stream(d), *self._id, self._type, self.page, q, table, lengths, scale, max_length)
            if made is not None:
                return made
        _, B, Hq, D, qt, qh = _heads(q, "q", _HALF, d)
        t = q.dtype
        if D != self.D or Hq == 0 or Hq % self.heads:
            raise ValueError(f"q has {Hq} heads of {D}; the cache has {self.heads} of {self.D}")
        if t != self.dtype and self.dtype in _HALF:
            raise ValueError(f"q has dtype {t}; the cache has {self.dtype}")
        at, W = self._table(table, B)
        lens = _vector(lengths, "lengths", _INT, B, d)
        bound = W * self.page
        if max_length is not None and max_length < bound:
            bound = max(int(max_length), 0)
        nb = lib.qmm_cache_attend_workspace_bytes(self._h, B, Hq, bound)
        if out is None:
            out = _empty((B, Hq, D), t, d)
        elif _out(out, (B, Hq, D), None, d).dtype != t:
            raise ValueError("out must have q's dtype")
        ws = torch.empty(nb, dtype=torch.uint8, device=q.device) if nb else None
        _call(d, lib.qmm_cache_attend, self._h, _pack_attend(
            q.data_ptr(), at, lens, out.data_ptr(), ws.data_ptr() if nb else 0, qt, qh, B, Hq, W, bound, nb, _HALF[t],
            D ** -0.5 if scale is None else _single(scale)))
        return out


def attend_prompt(q, k, v, starts, k_starts=None, causal=True, scale=None, out=None):
    """Attention of packed sequences: q [Tq, Hq, D], k and v [Tk, H, D] (fp16 or bf16; 16-byte aligned rows of k and v), Hq a
    multiple of H.  Sequence b has the queries from starts[b] and the keys from k_starts[b] on (int32 [B + 1], not
    decreasing; k_starts: starts by default).  causal: query i of n sees the keys 0 .. i + m - n of its m; one that sees
    none gives zeros.  Rows of no sequence are not written: they stay as they were in `out`."""
    d = _here(q)
    if out is None and d >= 0:
        made = _calls.attend_prompt(d, _current_stream(d), q, k, v, starts, k_starts, causal, scale)
        if made is not None:
            return made
    d, Tq, Hq, D, qt, qh = _heads(q, "q", _HALF)
    t = q.dtype
    _, Tk, H, Dk, kt, kh = _heads(k, "k", (t,), d)
    _, Tv, Hv, Dv, vt, vh = _heads(v, "v", (t,), d)
    if Dk != D or H == 0 or Hq == 0 or Hq % H:
        raise ValueError(f"k has {H} heads of {Dk}; q has {Hq} of {D}")
    if Tv != Tk or Hv != H or Dv != D:
        raise ValueError(f"v has shape {tuple(v.shape)}; k has {tuple(k.shape)}")
    _tensor(starts, "starts", (_INT,), (1,))
    n = starts.shape[0]
    if n < 1:
        raise ValueError("starts is empty")
    qs = _vector(starts, "starts", _INT, n, d)
    if k_starts is None or k_starts is starts:
        if Tk != Tq:
            raise ValueError(f"{Tk} keys for {Tq} queries need k_starts")
        ks = qs
    else:
        ks = _vector(k_starts, "k_starts", _INT, n, d)
    if out is None:
        out = _empty((Tq, Hq, D), t, d)
    elif _out(out, (Tq, Hq, D), None, d).dtype != t:
        raise ValueError("out must have q's dtype")
    _call(d, lib.qmm_attend_prompt, _pack_prompt(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, out.data_ptr(), qt, qh, kt, kh, vt, vh, n - 1, Tq, Tk, Hq, H, D, _HALF[t],
        1 if causal else 0, D ** -0.5 if scale is None else _single(scale)))
    return out
