"""The expert router and the sum of its slots: the binding of include/qmm.h's qmm_route* calls.

    r = route(logits, S, normalise=True, coef=0.01)      # ids, weights, counts, psum, loss
    y = experts.linear_id(x, r.ids)                      # F8Matrix, or QMatrix.gemm_id
    out = route_combine(y, r.weights)

Backward (no autograd: results carry no gradient history whatever their inputs require, every gradient is a call):

    dy, dweights = route_combine_backward(y, r.weights, dout)
    dlogits = route_backward(logits, r, dweights, dloss)

A trainer that adds counts and psum over GPUs before the loss calls balance_loss on the sums and hands a Routing with
the summed counts to route_backward.  Counts stay int32 (torch.sum of int32 gives int64, which both calls refuse: pass
dtype=torch.int32).
"""

from typing import NamedTuple, Optional

import torch

from ._lib import lib
from .f8 import _DT, _Seen, _call, _empty, _out, _place, _shape, _tensor


class Routing(NamedTuple):
    ids: torch.Tensor      # int32 [N, S], -1: no expert left
    weights: torch.Tensor  # fp32 [N, S]
    counts: torch.Tensor   # int32 [E + 1]: pairs per expert, then the rows that have an expert
    psum: torch.Tensor     # fp32 [E]: sum of the probabilities over the rows
    loss: torch.Tensor     # fp32, no dimension
    normalise: bool
    coef: float
    valid: Optional[torch.Tensor]


class RoutePlan:
    """(token, slot) pairs of ids [N, S] sorted by expert; see route_plan.  data is qmm_route_plan's buffer, int32, of
    these sizes: every call that reads it checks that it holds as much."""

    __slots__ = ("data", "N", "S", "n_experts", "routed", "bytes")

    def __init__(self, data, N, S, n_experts):
        _tensor(data, "data", (torch.int32,), (1,))
        self.data, self.N, self.S, self.n_experts = data, N, S, n_experts
        self.bytes, self.routed = _plan_size(N * S, n_experts)

    def place(self, device):
        """Pointer of the plan's buffer, which is as large as its sizes need and on device."""
        if self.data.numel() * 4 < self.bytes or self.bytes == 0:
            raise ValueError(f"the plan's data has {self.data.numel() * 4} bytes; {self.N} x {self.S} ids of {self.n_experts} "
                             f"experts need {self.bytes}")
        _place(device, (self.data, "plan"))
        return self.data.data_ptr()

    @property
    def counts(self):
        """Pairs per expert, int32 [E] (a view of the plan)."""
        return self.data[:self.n_experts]

    def per_slot(self, rows, name):
        """1: a row per (token, slot) pair, 0: a row per token."""
        if rows == self.N and self.S != 1:
            return 0
        if rows != self.N * self.S:
            raise ValueError(f"{name} has {rows} rows; the plan's ids are {self.N} x {self.S}")
        return 1

    def per_slot_rows(self, x, name):
        if x.dim() == 3:
            _shape(x, name, (self.N, self.S, x.shape[2]))
            return 1
        return self.per_slot(x.shape[0], name)


_plan_sizes = _Seen()  # of the pairs and experts seen


def _plan_size(pairs, E):
    """Bytes of a plan, tokens of a quantization along its pairs."""
    size = _plan_sizes.get((pairs, E))
    if size is None:
        size = _plan_sizes[pairs, E] = lib.qmm_route_plan_bytes(pairs, E), lib.qmm_f8_routed_tokens(pairs, E)
    return size


def route_plan(ids: torch.Tensor, n_experts: int) -> RoutePlan:
    """Sort the pairs of ids [N, S] (int32; -1: an empty slot) by expert, once for every product that reads them."""
    _tensor(ids, "ids", (torch.int32,), (2,))
    N, S = ids.shape
    E = int(n_experts)
    if S < 1 or E < 1:
        raise ValueError("ids needs a slot and the plan an expert")
    device = _place(None, (ids, "ids"))
    nb = _plan_size(N * S, E)[0]
    data = torch.empty(max(nb, 16) // 4, dtype=torch.int32, device=ids.device)
    _call(device, lib.qmm_route_plan, ids.data_ptr(), N, S, E, data.data_ptr(), nb)
    return RoutePlan(data, N, S, E)


def _logits(logits, valid):
    _tensor(logits, "logits", _DT, (2,))
    if valid is not None:
        _tensor(valid, "valid", (torch.uint8, torch.bool), (1,))
        _shape(valid, "valid", (logits.shape[0],))


def _place_logits(logits, valid, *named):
    if valid is not None:
        named += ((valid, "valid"),)
    return _place(None, (logits, "logits"), *named)


_route_need = _Seen()  # workspace bytes of the sizes seen


def route(logits: torch.Tensor, S: int, normalise: bool = True, coef: float = 0.0,
          valid: Optional[torch.Tensor] = None) -> Routing:
    """Softmax over logits [N, E], the S largest experts of each row and the balance loss.  valid [N] (uint8 or bool):
    0 marks padded rows."""
    _logits(logits, valid)
    device = _place_logits(logits, valid)
    N, E = logits.shape
    S = int(S)
    if not 1 <= S <= min(E, 64):
        raise ValueError(f"S={S} outside [1, {min(E, 64)}]")
    on = logits.device
    ids, weights = _empty((N, S), torch.int32, device), _empty((N, S), torch.float32, device)
    counts = torch.empty(E + 1, dtype=torch.int32, device=on)
    nb = _route_need.get((N, E))
    if nb is None:
        nb = _route_need[N, E] = lib.qmm_route_workspace_bytes(N, E)
    # sums over the rows, the loss and the workspace in one allocation
    pad = (E + 1 + 3) // 4 * 4
    buf = torch.empty(pad + nb // 4, dtype=torch.float32, device=on)
    psum, loss, at = buf.as_strided((E,), (1,)), buf.as_strided((), (), E), buf.data_ptr()
    _call(device, lib.qmm_route, logits.data_ptr(), _DT[logits.dtype], N, E, S,
          valid.data_ptr() if valid is not None else None, int(bool(normalise)), coef, ids.data_ptr(), weights.data_ptr(),
          counts.data_ptr(), at, at + 4 * E, at + 4 * pad, nb)
    return Routing(ids, weights, counts, psum, loss, bool(normalise), float(coef), valid)


def balance_loss(counts: torch.Tensor, psum: torch.Tensor, S: int, coef: float) -> torch.Tensor:
    """coef * sum_e f_e P_e from counts [E + 1] and psum [E] (added over micro-batches or GPUs)."""
    _tensor(counts, "counts", (torch.int32,), (1,))
    _tensor(psum, "psum", (torch.float32,), (1,))
    E = psum.shape[0]
    _shape(counts, "counts", (E + 1,))
    device = _place(None, (counts, "counts"), (psum, "psum"))
    loss = torch.empty((), dtype=torch.float32, device=counts.device)
    _call(device, lib.qmm_balance_loss, counts.data_ptr(), psum.data_ptr(), E, int(S), float(coef), loss.data_ptr())
    return loss


def route_backward(logits: torch.Tensor, routing: Routing, dweights: Optional[torch.Tensor] = None,
                   dloss: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dlogits [N, E] of logits' type from the gradients with respect to the weights ([N, S] fp32) and the loss (fp32, one
    element on the device); either may be None.  ids and counts are int32, as route gives them."""
    ids, _, counts, _, _, normalise, coef, valid = routing
    _logits(logits, valid)
    _tensor(ids, "ids", (torch.int32,), (2,))
    _tensor(counts, "counts", (torch.int32,), (1,))
    N, E = logits.shape
    S = ids.shape[1]
    _shape(ids, "ids", (N, S))
    _shape(counts, "counts", (E + 1,))
    device = _place_logits(logits, valid, (ids, "ids"), (counts, "counts"))
    if dweights is not None:
        _tensor(dweights, "dweights", (torch.float32,), (2,))
        _shape(dweights, "dweights", (N, S))
        _place(device, (dweights, "dweights"))
    if dloss is not None:
        _tensor(dloss, "dloss", (torch.float32,))
        if dloss.numel() != 1:
            raise ValueError("dloss must have one element")
        _place(device, (dloss, "dloss"))
    dlogits = torch.empty_like(logits)
    _call(device, lib.qmm_route_backward, logits.data_ptr(), _DT[logits.dtype], N, E, S,
          valid.data_ptr() if valid is not None else None, int(normalise), coef, ids.data_ptr(),
          dweights.data_ptr() if dweights is not None else None, counts.data_ptr(),
          dloss.data_ptr() if dloss is not None else None, dlogits.data_ptr())
    return dlogits


def _slots(y, weights):
    _tensor(y, "y", _DT, (3,))
    device = _place(None, (y, "y"))
    N, S, M = y.shape
    if S < 1 or M < 1:
        raise ValueError("y needs a slot and a column")
    if weights is not None:
        _tensor(weights, "weights", (torch.float32, y.dtype), (2,))
        _shape(weights, "weights", (N, S))
        _place(device, (weights, "weights"))
    return device, N, S, M


def route_combine(y: torch.Tensor, weights: Optional[torch.Tensor] = None, out: torch.Tensor = None) -> torch.Tensor:
    """out [N, M] = sum over the slots of weights [N, S] (fp32 or y's type) times y [N, S, M]; without weights the plain
    sum (the gradient of a row that a token's slots share).  A slot of weight 0 adds nothing, whatever its row holds."""
    device, N, S, M = _slots(y, weights)
    o = _out(out, (N, M), y.dtype, device)
    if o.dtype != y.dtype:
        raise ValueError("out must have y's dtype")
    _call(device, lib.qmm_route_combine, y.data_ptr(), _DT[y.dtype], weights.data_ptr() if weights is not None else None,
          _DT[weights.dtype] if weights is not None else 0, N, S, M, o.data_ptr())
    return o


def route_combine_backward(y: torch.Tensor, weights: torch.Tensor, dout: torch.Tensor):
    """(dy [N, S, M] of y's type, dweights [N, S] of weights' type) from dout [N, M] of y's type."""
    if weights is None:
        raise ValueError("weights are needed; without them dy is dout for every slot")
    device, N, S, M = _slots(y, weights)
    _tensor(dout, "dout", (y.dtype,), (2,))
    _shape(dout, "dout", (N, M))
    _place(device, (dout, "dout"))
    dy, dw = torch.empty_like(y), torch.empty_like(weights)
    _call(device, lib.qmm_route_combine_backward, y.data_ptr(), _DT[y.dtype], weights.data_ptr(), _DT[weights.dtype], N, S, M,
          dout.data_ptr(), dy.data_ptr(), dw.data_ptr())
    return dy, dw
