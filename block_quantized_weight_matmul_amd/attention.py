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

import torch

from ._lib import check, lib
from .f8 import _DT, _call, _empty, _out, _place, _shape, _tensor

_HALF = (torch.float16, torch.bfloat16)
_CACHE = {torch.float16: 1, torch.bfloat16: 2, torch.uint8: 3, torch.float8_e4m3fn: 3}
_I32 = (torch.int32,)
_F32 = (torch.float32,)


def _heads(x, name, dtypes, device=None):
    """(device, T, heads, D, stride of a token, stride of a head) of a [T, heads, D] device tensor."""
    _tensor(x, name, dtypes, (3,))
    d = x.get_device()
    if d < 0:
        raise ValueError(f"{name} must be a device tensor")
    if device is not None and d != device:
        raise ValueError(f"{name} is on cuda:{d}; expected cuda:{device}")
    T, H, D = x.shape
    st, sh, step = x.stride()
    if step != 1 and D > 1:
        raise ValueError(f"{name} must have a contiguous last axis")
    return d, T, H, D, st, sh


def _vector(t, name, dtypes, length, device):
    _tensor(t, name, dtypes, (1,))
    if t.shape[0] != length:
        raise ValueError(f"{name} has {t.shape[0]} elements; expected {length}")
    _place(device, (t, name))
    return t.data_ptr()


def _rotation(positions, inv_freq, T, device):
    if inv_freq is None:
        return None, None, 0
    if positions is None:
        raise ValueError("inv_freq needs positions")
    _tensor(inv_freq, "inv_freq", _F32, (1,))
    n = inv_freq.shape[0]
    return _vector(positions, "positions", _I32, T, device), _vector(inv_freq, "inv_freq", _F32, n, device), 2 * n


def _weights(q_weight, k_weight, D, device):
    first = q_weight if q_weight is not None else k_weight
    if first is None:
        return None, None, 0
    dtypes = _DT if q_weight is None or k_weight is None else (first.dtype,)
    _tensor(first, "q_weight" if q_weight is not None else "k_weight", _DT)
    return tuple(None if w is None else _vector(w, name, dtypes, D, device)
                 for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight"))) + (_DT[first.dtype],)


def head_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, dtype=None):
    """(q', k'): every head of q [T, Hq, D] and k [T, H, D] divided by its root mean square and multiplied by its weight [D]
    (None: no norm), then its first 2 len(inv_freq) columns rotated by positions [T] (int32) times inv_freq (fp32; None: no
    rotation), column i with column i + len(inv_freq), or 2 i with 2 i + 1 where interleaved.  dtype: of the results."""
    device, T, Hq, D, qt, qh = _heads(q, "q", _DT)
    _, Tk, H, Dk, kt, kh = _heads(k, "k", (q.dtype,), device)
    if Tk != T or Dk != D:
        raise ValueError(f"k has shape {tuple(k.shape)}; q has {tuple(q.shape)}")
    dtype = q.dtype if dtype is None else dtype
    _tensor_type(dtype)
    pos, freq, R = _rotation(positions, inv_freq, T, device)
    qw, kw, wt = _weights(q_weight, k_weight, D, device)
    qo, ko = _empty((T, Hq, D), dtype, device), _empty((T, H, D), dtype, device)
    _call(device, lib.qmm_head_norm_rope, q.data_ptr(), qt, qh, k.data_ptr(), kt, kh, _DT[q.dtype], T, Hq, H, D, qw, kw, wt,
          eps, pos, freq, R, int(bool(interleaved)), qo.data_ptr(), ko.data_ptr(), _DT[dtype])
    return qo, ko


def _tensor_type(dtype):
    if dtype not in _DT:
        raise ValueError(f"dtype {dtype}; expected one of {[str(d) for d in _DT]}")


class KVCache:
    """A paged cache of keys and values, k and v [pages, heads, page, D]: fp16, bf16, or e4m3 codes (uint8 or float8_e4m3fn)
    with fp32 scales [pages, heads, page], one per token and head.  page is a power of two from 16 on, D a multiple of 16 up
    to 256.  The tensors are kept referenced and written in place.

    A token's slot is its page times `page` plus its row there; a table int32 [B, W] names the pages of B sequences in
    order, entries past a sequence's last page are not read."""

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
        self._sizes = {}
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            check(lib.qmm_cache_create(ctypes.byref(h), *(t.data_ptr() for t, _ in named), *([None] * (4 - len(named))),
                                       _CACHE[k.dtype], self.pages, self.page, self.heads, self.D))
        self._h = h

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

    def _kv(self, k, v, device):
        _, T, H, D, kt, kh = _heads(k, "k", _DT, device)
        _, Tv, Hv, Dv, vt, vh = _heads(v, "v", (k.dtype,), device)
        if (H, D) != (self.heads, self.D):
            raise ValueError(f"k has {H} heads of {D}; the cache has {self.heads} of {self.D}")
        if (Tv, Hv, Dv) != (T, H, D):
            raise ValueError(f"v has shape {tuple(v.shape)}; k has {tuple(k.shape)}")
        return T, (k.data_ptr(), kt, kh, v.data_ptr(), vt, vh)

    def write(self, k, v, slots):
        """k and v [T, heads, D] to slots [T] (int32; negative ones and those past the last page are left out).  The slots
        of a call are distinct."""
        T, rows = self._kv(k, v, self.device)
        at = _vector(slots, "slots", _I32, T, self.device)
        _call(self.device, lib.qmm_cache_write, self._h, *rows, _DT[k.dtype], T, at)

    def norm_rope_write(self, q, k, v, slots, positions, inv_freq, q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                        dtype=None):
        """head_norm_rope of q and k, then write of the keys and of v, in one launch and with the same bits; returns q'.
        dtype: of q' and, before they are quantized, of the keys; the cache's own unless that is e4m3 (then q's)."""
        d = self.device
        _, T, Hq, D, qt, qh = _heads(q, "q", _DT, d)
        Tk, rows = self._kv(k, v, d)
        if k.dtype != q.dtype:
            raise ValueError(f"k has dtype {k.dtype}; q has {q.dtype}")
        if Tk != T or D != self.D:
            raise ValueError(f"q has shape {tuple(q.shape)}; k has {tuple(k.shape)}")
        if dtype is None:
            dtype = self.dtype if self.dtype in _HALF else q.dtype
        _tensor_type(dtype)
        if self.dtype in _HALF and dtype != self.dtype:
            raise ValueError(f"dtype {dtype}; the cache has {self.dtype}")
        pos, freq, R = _rotation(positions, inv_freq, T, d)
        qw, kw, wt = _weights(q_weight, k_weight, D, d)
        at = _vector(slots, "slots", _I32, T, d)
        o = _empty((T, Hq, D), dtype, d)
        _call(d, lib.qmm_cache_norm_rope_write, self._h, q.data_ptr(), qt, qh, *rows, _DT[q.dtype], T, Hq, qw, kw, wt, eps, pos,
              freq, R, int(bool(interleaved)), at, o.data_ptr(), _DT[dtype])
        return o

    def _table(self, table, B):
        _tensor(table, "table", _I32, (2,))
        if table.shape[0] != B:
            raise ValueError(f"table has {table.shape[0]} rows; expected {B}")
        _place(self.device, (table, "table"))
        return table.data_ptr(), table.shape[1]

    def read(self, table, starts, total, dtype=None, out=None):
        """(k, v) [total, heads, D]: sequence b's tokens as rows starts[b] .. starts[b + 1] - 1 (starts int32 [B + 1], not
        decreasing).  Rows of no sequence are not written: they stay as they were in `out`, a pair of tensors."""
        _tensor(starts, "starts", _I32, (1,))
        B = starts.shape[0] - 1
        if B < 0:
            raise ValueError("starts is empty")
        at, W = self._table(table, B)
        _place(self.device, (starts, "starts"))
        total = int(total)
        if total < 0:
            raise ValueError(f"total={total} is negative")
        shape = (total, self.heads, self.D)
        if out is None:
            dtype = (self.dtype if self.dtype in _HALF else torch.bfloat16) if dtype is None else dtype
            _tensor_type(dtype)
            k, v = _empty(shape, dtype, self.device), _empty(shape, dtype, self.device)
        else:
            k, v = out
            _out(k, shape, None, self.device, "out[0]")
            _out(v, shape, None, self.device, "out[1]")
            if v.dtype != k.dtype or dtype not in (None, k.dtype):
                raise ValueError("out must be two tensors of one dtype, that of the call")
        _call(self.device, lib.qmm_cache_read, self._h, at, B, W, starts.data_ptr(), total, k.data_ptr(), v.data_ptr(),
              _DT[k.dtype])
        return k, v

    def attend(self, q, table, lengths, scale=None, max_length=None, out=None):
        """Attention of one token per sequence, q [B, Hq, D] (fp16 or bf16, a 16-bit cache's own type), over the first
        lengths[b] (int32) tokens of each sequence; Hq a multiple of the cache's heads.  scale: of the scores, 1 / sqrt(D) by
        default.  max_length: the longest length where the host knows it, else the table's reach; it decides how the work
        is divided and nothing else."""
        d = self.device
        _, B, Hq, D, qt, qh = _heads(q, "q", _HALF, d)
        if D != self.D or Hq == 0 or Hq % self.heads:
            raise ValueError(f"q has {Hq} heads of {D}; the cache has {self.heads} of {self.D}")
        if self.dtype in _HALF and q.dtype != self.dtype:
            raise ValueError(f"q has dtype {q.dtype}; the cache has {self.dtype}")
        at, W = self._table(table, B)
        lens = _vector(lengths, "lengths", _I32, B, d)
        reach = W * self.page
        bound = reach if max_length is None else min(max(int(max_length), 0), reach)
        key = B, Hq, bound
        nb = self._sizes.get(key)
        if nb is None:
            if len(self._sizes) >= 1024:
                self._sizes.clear()
            nb = self._sizes[key] = lib.qmm_cache_attend_workspace_bytes(self._h, B, Hq, bound)
        o = _out(out, (B, Hq, D), q.dtype, d)
        if o.dtype != q.dtype:
            raise ValueError("out must have q's dtype")
        ws = torch.empty(nb, dtype=torch.uint8, device=o.device) if nb else None
        _call(d, lib.qmm_cache_attend, self._h, q.data_ptr(), _DT[q.dtype], qt, qh, B, Hq, at, W, lens, bound,
              D ** -0.5 if scale is None else scale, o.data_ptr(), ws.data_ptr() if nb else None, nb)
        return o


def attend_prompt(q, k, v, starts, k_starts=None, causal=True, scale=None, out=None):
    """Attention of packed sequences: q [Tq, Hq, D], k and v [Tk, H, D] (fp16 or bf16; 16-byte aligned rows of k and v), Hq a
    multiple of H.  Sequence b has the queries from starts[b] and the keys from k_starts[b] on (int32 [B + 1], not
    decreasing; k_starts: starts by default).  causal: query i of n sees the keys 0 .. i + m - n of its m; one that sees
    none gives zeros.  Rows of no sequence are not written: they stay as they were in `out`."""
    d, Tq, Hq, D, qt, qh = _heads(q, "q", _HALF)
    _, Tk, H, Dk, kt, kh = _heads(k, "k", (q.dtype,), d)
    _, Tv, Hv, Dv, vt, vh = _heads(v, "v", (q.dtype,), d)
    if Dk != D or H == 0 or Hq == 0 or Hq % H:
        raise ValueError(f"k has {H} heads of {Dk}; q has {Hq} of {D}")
    if (Tv, Hv, Dv) != (Tk, H, Dk):
        raise ValueError(f"v has shape {tuple(v.shape)}; k has {tuple(k.shape)}")
    k_starts = starts if k_starts is None else k_starts
    _tensor(starts, "starts", _I32, (1,))
    n = starts.shape[0]
    if n < 1:
        raise ValueError("starts is empty")
    if k_starts is starts and Tk != Tq:
        raise ValueError(f"{Tk} keys for {Tq} queries need k_starts")
    qs, ks = _vector(starts, "starts", _I32, n, d), _vector(k_starts, "k_starts", _I32, n, d)
    o = _out(out, (Tq, Hq, D), q.dtype, d)
    if o.dtype != q.dtype:
        raise ValueError("out must have q's dtype")
    _call(d, lib.qmm_attend_prompt, q.data_ptr(), qt, qh, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, _DT[q.dtype], qs, ks,
          n - 1, Tq, Tk, Hq, H, D, int(bool(causal)), D ** -0.5 if scale is None else scale, o.data_ptr())
    return o
