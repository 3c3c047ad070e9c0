"""Measured cases of the library's block-of-128 e4m3 products and of the expert router.

Kinds of case (sizes: the decode-layer and expert shapes of qmm_synth.workloads, and generic odd ones):

``linear``        y = x W^T with W stored as e4m3 codes and one scale per 128 x 128 block; the tokens are
                  quantized in the call, one scale per token and 128 values along K.  Serving.
``linear_train``  the same product in training: weights (fp32 masters), tokens and output gradients are
                  quantized in the step, which gives y, dx = dy W and dW = dy^T x, all of the tokens' type.
``experts``       the product with an expert's matrix picked for every (token, slot).
``experts_train`` expert products, their weighted sum per token, and the gradients of all of it.
``route``         a router: softmax over the experts, the S largest, their weights, tokens per expert and the
                  balance loss; with ``train`` the gradient with respect to the logits too.

An id of -1 is an empty slot (a dropped or padded token): no product, a row of zeros, no gradient.
"""

import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -80  # smallest scale of a block (an all-zero block has it)
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
WEIGHT_STD = 0.02
BALANCE_COEF = 0.01


# ---- cases -------------------------------------------------------------------------------------

def listed():
    return [
        # the query projection of one decoded token
        dict(name="linear_q_1", kind="linear", N=1, M=4096, K=2560, dtype="bf16", strided=False),
        # the down projection of a batch of 16 decoded sequences
        dict(name="linear_down_16", kind="linear", N=16, M=2560, K=9728, dtype="f16", strided=False),
        # odd everything, tokens sliced out of a wider buffer: ragged blocks along M, N and K
        dict(name="linear_odd_333", kind="linear", N=333, M=1000, K=1111, dtype="f32", strided=True),
        # the gate projection of a 2048-token prefill
        dict(name="linear_gate_2048", kind="linear", N=2048, M=9728, K=2560, dtype="bf16", strided=False),
        # a training step of the query projection on 4096 tokens
        dict(name="train_q_4096", kind="linear_train", N=4096, M=4096, K=2560, dtype="bf16"),
        # a training step where no size is a multiple of the block
        dict(name="train_odd_777", kind="linear_train", N=777, M=1300, K=515, dtype="f32"),
        # the down projection of 128 experts for four decoded tokens of eight slots each
        dict(name="experts_decode_4", kind="experts", N=4, S=8, E=128, M=4096, K=512, dtype="f32", per_slot=True,
             empty=0.0),
        # the up projection of the same experts for a 2048-token prefill: slots share their token's row
        dict(name="experts_prefill_2048", kind="experts", N=2048, S=8, E=128, M=4096, K=512, dtype="bf16",
             per_slot=False, empty=0.0),
        # a training step of eight large experts
        dict(name="experts_train_2048", kind="experts_train", N=2048, S=2, E=8, M=2048, K=2560, dtype="bf16",
             empty=0.0),
        # ragged experts with dropped slots
        dict(name="experts_train_odd", kind="experts_train", N=391, S=3, E=24, M=520, K=776, dtype="f32", empty=0.1),
        # the router of a decode step
        dict(name="route_decode_16", kind="route", N=16, E=128, S=8, dtype="f32", normalise=True, masked=0.0,
             train=False),
        # the router of a training step, with experts masked out and rows that are padding
        dict(name="route_train_16384", kind="route", N=16384, E=128, S=8, dtype="bf16", normalise=True, masked=0.2,
             train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["linear", "linear", "linear_train", "experts", "experts_train", "route"])
    dtype = rng.choice(sorted(DTYPES))
    if kind == "route":
        E = _log(rng, 8, 512)
        return dict(kind=kind, N=_log(rng, 1, 16384), E=E, S=rng.randint(1, min(8, E)), dtype=dtype,
                    normalise=rng.random() < 0.5, masked=rng.choice([0.0, 0.2]), train=rng.random() < 0.5)
    if kind in ("linear", "linear_train"):
        most = 1.0e11 if kind == "linear" else 4.0e10
        N, M, K = _log(rng, 1, 4096), _log(rng, 64, 9728), _log(rng, 64, 9728)
        N = max(1, min(N, int(most / (2.0 * M * K))))
        case = dict(kind=kind, N=N, M=M, K=K, dtype=dtype)
        if kind == "linear":
            case["strided"] = rng.random() < 0.5
        return case
    E = _log(rng, 4, 128)
    M, K = _log(rng, 64, 4096), _log(rng, 64, 2560)
    if E * M * K > 2.0e8:
        M = max(64, int(2.0e8 / (E * K)))
    S = rng.randint(1, min(8, E))
    N = _log(rng, 1, 2048)
    N = max(1, min(N, int(2.0e10 / (2.0 * S * M * K))))
    case = dict(kind=kind, N=N, S=S, E=E, M=M, K=K, dtype=dtype, empty=rng.choice([0.0, 0.1]))
    if kind == "experts":
        case["per_slot"] = rng.random() < 0.5
    return case


def _padded(n):
    return -(-n // BLOCK) * BLOCK


def work(case):
    kind, N = case["kind"], case["N"]
    b = DTYPES[case["dtype"]].itemsize
    if kind == "route":
        E, S = case["E"], case["S"]
        passes = 2 if case["train"] else 1
        return {"bytes": float(passes * N * E * b + N * S * (8 + (4 if case["train"] else 0)) + 8 * E),
                "flops": float(passes * 6 * N * E)}
    M, K = case["M"], case["K"]
    codes = M * _padded(K) + 4 * (_padded(M) // BLOCK) * (_padded(K) // BLOCK)
    if kind == "linear":
        return {"bytes": float(N * K * b + codes + N * M * b), "flops": 2.0 * N * M * K}
    if kind == "linear_train":
        return {"bytes": float(2 * N * K * b + 2 * N * M * b + (4 + b) * M * K), "flops": 6.0 * N * M * K}
    S, E = case["S"], case["E"]
    pairs = N * S * (1.0 - case["empty"])
    if kind == "experts":
        rows = pairs if case["per_slot"] else N
        used = E * (1.0 - (1.0 - S / E) ** N)
        return {"bytes": float(rows * K * b + used * codes + N * S * M * b), "flops": 2.0 * pairs * M * K}
    return {"bytes": float(2 * N * K * b + 2 * N * M * b + (4 + b) * E * M * K + (4 + 2 * b) * N * S),
            "flops": 6.0 * pairs * M * K}


# ---- inputs ------------------------------------------------------------------------------------

def _activations(g, rows, K, dtype):
    """N(0, 1) with every 64th channel eight times larger, as hidden states have."""
    x = torch.randn((rows, K), generator=g, device="cuda")
    x[:, ::64] *= 8.0
    return x.to(dtype)


def _expert_ids(g, N, S, E, empty):
    """S distinct experts a token, some experts more popular than others, a share of the slots empty."""
    liking = torch.rand((1, E), generator=g, device="cuda") * 0.5
    ids = (torch.rand((N, E), generator=g, device="cuda") + liking).topk(S, dim=1).indices.to(torch.int32)
    if empty:
        ids = torch.where(torch.rand((N, S), generator=g, device="cuda") < empty, torch.full_like(ids, -1), ids)
    return ids


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    kind, N, dtype = case["kind"], case["N"], DTYPES[case["dtype"]]
    s = dict(case=dict(case))
    if kind == "route":
        E = case["E"]
        logits = torch.randn((N, E), generator=g, device="cuda") * 1.5 + torch.randn((1, E), generator=g, device="cuda")
        if case["masked"]:
            off = torch.rand((N, E), generator=g, device="cuda") < case["masked"]
            off |= torch.rand((N, 1), generator=g, device="cuda") < case["masked"] / 8  # rows that leave nothing
            logits = logits.masked_fill(off, float("-inf"))
        s["logits"] = logits.to(dtype)
        s["dweights"] = torch.randn((N, case["S"]), generator=g, device="cuda") * 1e-3
        s["dloss"] = torch.ones((), device="cuda")
        return s
    M, K = case["M"], case["K"]
    if kind in ("linear", "linear_train"):
        wide = K + 24 if case.get("strided") else K
        s["x"] = _activations(g, N, wide, dtype)[:, :K]
        w = torch.randn((1, M, K), generator=g, device="cuda") * WEIGHT_STD
    else:
        E, S = case["E"], case["S"]
        s["ids"] = _expert_ids(g, N, S, E, case["empty"])
        s["x"] = _activations(g, N * S, K, dtype).view(N, S, K) if case.get("per_slot") else _activations(g, N, K, dtype)
        w = torch.randn((E, M, K), generator=g, device="cuda") * WEIGHT_STD
        # rows of the fullest expert, for the plain form's batched products
        s["capacity"] = _padded(max(1, int(torch.bincount((s["ids"].flatten() + 1).long(), minlength=E + 1)[1:].max())))
    if kind.endswith("train"):
        s["w"] = w if kind == "experts_train" else w[0]
        s["dy"] = (torch.randn((N, M), generator=g, device="cuda") * 1e-3).to(dtype)
        if kind == "experts_train":
            s["weights"] = torch.softmax(torch.randn((N, S), generator=g, device="cuda"), dim=1).to(dtype)
    else:
        values, scales = _quantize_weight(w)
        s["codes"], s["scales"] = _codes(values), scales
        if kind == "linear":
            s["codes"], s["scales"] = s["codes"][0], s["scales"][0]
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import block_quantized_weight_matmul_amd as q
        kind = case["kind"]
        if kind in ("linear", "experts"):
            s["matrix"] = q.F8Matrix(s["codes"], s["scales"], case["M"], case["K"], case.get("E", 1))
        elif kind.endswith("train"):
            # the buffers a trainer keeps: the codes of the weights and of their transpose
            s["matrix"] = q.F8Matrix.quantize(s["w"])
            s["matrix_t"] = s["matrix"].transposed()
    return s


# ---- the plain forms ---------------------------------------------------------------------------

def _e4m3(v):
    """Nearest e4m3 value (ties to even) of the float64 v, |v| <= 448."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(e - 1, min=-6) - 3)
    return torch.round(v / step) * step


def _scale(amax):
    """amax / 448 rounded to fp32 (the quotient in 64 bits: a product with 1 / 448 would miss it by a step)."""
    return torch.clamp((amax.double() / E4M3_MAX).float(), min=MIN_SCALE)


def _quantize(x):
    """One scale per 128 values of the last axis: values [..., padded] fp32, scales [..., groups] fp32."""
    x = torch.nn.functional.pad(x.float(), (0, _padded(x.shape[-1]) - x.shape[-1]))
    b = x.unflatten(-1, (-1, BLOCK))
    s = _scale(b.abs().amax(-1))
    return _e4m3(b.double() / s.double().unsqueeze(-1)).float().flatten(-2), s


def _quantize_weight(w):
    """One scale per 128 x 128 block of [E, M, K]: values [E, M, padded K], scales [E, blocks of M, blocks of K]."""
    E, M, K = w.shape
    w = torch.nn.functional.pad(w.float(), (0, _padded(K) - K, 0, _padded(M) - M))
    b = w.view(E, _padded(M) // BLOCK, BLOCK, _padded(K) // BLOCK, BLOCK)
    s = _scale(b.abs().amax((2, 4)))
    values = _e4m3(b.double() / s.double()[:, :, None, :, None]).float()
    return values.reshape(E, _padded(M), _padded(K))[:, :M].contiguous(), s


def _codes(values):
    return values.to(torch.float8_e4m3fn).view(torch.uint8)


def _values(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _spread(values, scales):
    """values [..., padded] times their group's scale."""
    return (values.unflatten(-1, (-1, BLOCK)) * scales.unsqueeze(-1)).flatten(-2)


def _spread_weight(values, scales):
    M, K = values.shape[-2:]
    full = scales.repeat_interleave(BLOCK, -2)[..., :M, :].repeat_interleave(BLOCK, -1)[..., :K]
    return values * full


def _plain_linear(s):
    x = s["x"]
    xd = _spread(*_quantize(x))
    wd = _spread_weight(_values(s["codes"]), s["scales"])
    return (xd @ wd.t()).to(x.dtype)


def _plain_linear_train(s):
    x, dy, w, c = s["x"], s["dy"], s["w"], s["case"]
    M, K = c["M"], c["K"]
    values, scales = _quantize_weight(w[None])
    wd = _spread_weight(values, scales)[0]
    y = _spread(*_quantize(x)) @ wd.t()
    dx = _spread(*_quantize(dy))[:, :M] @ wd[:, :K]
    dw = _spread(*_quantize(dy.t())) @ _spread(*_quantize(x.t())).t()
    return {"y": y.to(x.dtype), "dx": dx.to(x.dtype), "dw": dw.to(x.dtype)}


def _dispatch(ids, E, capacity):
    """Row of every pair in [E * capacity] (the experts' pairs in order); empty slots go to one spare row."""
    flat = ids.flatten().long()
    mine = torch.nn.functional.one_hot(flat + 1, E + 1)[:, 1:]
    place = (mine.cumsum(0) * mine).sum(1) - 1
    return torch.where(flat < 0, torch.full_like(flat, E * capacity), flat * capacity + place)


def _to_experts(rows, at, E, capacity):
    room = torch.zeros((E * capacity + 1, rows.shape[-1]), device=rows.device, dtype=rows.dtype)
    room[at] = rows
    room[-1] = 0
    return room[:-1].view(E, capacity, rows.shape[-1])


def _from_experts(y, at):
    y = y.flatten(0, 1)
    return torch.cat([y, torch.zeros_like(y[:1])])[at]


def _pair_rows(x, N, S):
    return x.reshape(N * S, x.shape[-1]) if x.dim() == 3 else x.repeat_interleave(S, 0)


def _plain_experts(s):
    x, c = s["x"], s["case"]
    N, S, E, M = c["N"], c["S"], c["E"], c["M"]
    at = _dispatch(s["ids"], E, s["capacity"])
    xe = _to_experts(_pair_rows(_spread(*_quantize(x)), N, S), at, E, s["capacity"])
    wd = _spread_weight(_values(s["codes"]), s["scales"])
    y = torch.bmm(xe, wd.transpose(1, 2).contiguous())
    return _from_experts(y, at).view(N, S, M).to(x.dtype)


def _plain_experts_train(s):
    x, dout, w, weights, c = s["x"], s["dy"], s["w"], s["weights"], s["case"]
    N, S, E, M, K, C = c["N"], c["S"], c["E"], c["M"], c["K"], s["capacity"]
    at = _dispatch(s["ids"], E, C)
    values, scales = _quantize_weight(w)
    wd = _spread_weight(values, scales)
    xe = _to_experts(_pair_rows(_spread(*_quantize(x)), N, S), at, E, C)
    y = _from_experts(torch.bmm(xe, wd.transpose(1, 2).contiguous()), at).view(N, S, M).to(x.dtype)
    out = (weights.float()[:, :, None] * y.float()).sum(1).to(x.dtype)
    dweights = (y.float() * dout.float()[:, None, :]).sum(2).to(weights.dtype)
    dpairs = (weights.float()[:, :, None] * dout.float()[:, None, :]).to(x.dtype).view(N * S, M)
    ge = _to_experts(_spread(*_quantize(dpairs)), at, E, C)[..., :M]
    dx = _from_experts(torch.bmm(ge.contiguous(), wd[..., :K].contiguous()), at).view(N, S, K).to(x.dtype)
    dx = dx.float().sum(1).to(x.dtype)
    gt = _spread(*_quantize(_to_experts(dpairs.float(), at, E, C).transpose(1, 2)))
    xt = _spread(*_quantize(_to_experts(_pair_rows(x, N, S).float(), at, E, C).transpose(1, 2)))
    dw = torch.bmm(gt, xt.transpose(1, 2).contiguous()).to(x.dtype)
    return {"out": out, "dx": dx, "dw": dw, "dweights": dweights}


def _plain_route(s):
    logits, c = s["logits"].float(), s["case"]
    N, E, S = c["N"], c["E"], c["S"]
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    ids, some = ids[:, :S], top[:, :S] > float("-inf")
    alive = some[:, :1]
    ex = torch.where(alive, torch.exp(logits - torch.where(alive, top[:, :1], torch.zeros_like(top[:, :1]))), 0.0)
    p = ex / torch.where(alive, ex.sum(1, keepdim=True), torch.ones_like(top[:, :1]))
    chosen = torch.where(some, p.gather(1, ids), 0.0)
    total = torch.where(alive, chosen.sum(1, keepdim=True), torch.ones_like(top[:, :1]))
    weights = chosen / total if c["normalise"] else chosen
    tokens = alive.sum()
    counts = torch.zeros(E, dtype=torch.int64, device=logits.device)
    counts = counts.index_add(0, ids.flatten(), some.flatten().to(torch.int64))
    share = torch.where(tokens > 0, counts.float() * E / (S * tokens.clamp(min=1)), 0.0)
    psum = p.sum(0)
    loss = BALANCE_COEF * (share * psum).sum() / tokens.clamp(min=1)
    got = {"ids": torch.where(some, ids, -1).to(torch.int32), "weights": weights,
           "counts": torch.cat([counts, tokens[None]]).to(torch.int32), "loss": loss}
    if c["train"]:
        dw = s["dweights"]
        if c["normalise"]:
            dchosen = (dw - (dw * weights).sum(1, keepdim=True)) / total
        else:
            dchosen = dw
        dp = (s["dloss"] * BALANCE_COEF / tokens.clamp(min=1)) * share[None, :].expand(N, E)
        dp = dp.scatter_add(1, ids, torch.where(some, dchosen, 0.0))
        got["dlogits"] = (p * (dp - (p * dp).sum(1, keepdim=True))).to(s["logits"].dtype)
    return got


# ---- the library's calls -----------------------------------------------------------------------

def _own_linear(s):
    return s["matrix"].linear(s["x"])


def _own_linear_train(s):
    import block_quantized_weight_matmul_amd as q
    x, dy, m, mt = s["x"], s["dy"], s["matrix"], s["matrix_t"]
    m.update(s["w"], transposed=mt)
    xq, xt = q.f8_quantize_pair(x)
    gq, gt = q.f8_quantize_pair(dy)
    return {"y": m.gemm(xq, out_dtype=x.dtype), "dx": mt.gemm(gq, out_dtype=x.dtype), "dw": q.f8_wgrad(gt, xt, dtype=x.dtype)}


def _own_experts(s):
    return s["matrix"].linear_id(s["x"], s["ids"])


def _own_experts_train(s):
    import block_quantized_weight_matmul_amd as q
    x, dout, ids, weights, m, mt = s["x"], s["dy"], s["ids"], s["weights"], s["matrix"], s["matrix_t"]
    m.update(s["w"], transposed=mt)
    plan = q.route_plan(ids, m.n_experts)
    y = m.gemm_id(q.f8_quantize(x), plan, out_dtype=x.dtype)
    out = q.route_combine(y, weights)
    dpairs, dweights = q.route_combine_backward(y, weights, dout)
    dx = q.route_combine(mt.gemm_id(q.f8_quantize(dpairs), plan, out_dtype=x.dtype))
    dw = q.f8_wgrad(q.f8_quantize_t(dpairs, plan), q.f8_quantize_t(x, plan), plan, dtype=x.dtype)
    return {"out": out, "dx": dx, "dw": dw, "dweights": dweights}


def _own_route(s):
    import block_quantized_weight_matmul_amd as q
    c = s["case"]
    r = q.route(s["logits"], c["S"], normalise=c["normalise"], coef=BALANCE_COEF)
    got = {"ids": r.ids, "weights": r.weights, "counts": r.counts, "loss": r.loss}
    if c["train"]:
        got["dlogits"] = q.route_backward(s["logits"], r, s["dweights"], s["dloss"])
    return got


def run(state):
    kind = state["case"]["kind"]
    if kind == "linear":
        return _own_linear(state) if own else _plain_linear(state)
    if kind == "linear_train":
        return _own_linear_train(state) if own else _plain_linear_train(state)
    if kind == "experts":
        return _own_experts(state) if own else _plain_experts(state)
    if kind == "experts_train":
        return _own_experts_train(state) if own else _plain_experts_train(state)
    return _own_route(state) if own else _plain_route(state)


# ---- the definitions in 64 bits ----------------------------------------------------------------
# Stored tensors keep their types: scales are fp32, codes e4m3, and where a step hands a tensor of the
# inputs' type to the next one, it is rounded to that type.

def _grid64(device):
    """The non-negative e4m3 values in order: code n of 127."""
    n = torch.arange(127, device=device, dtype=torch.float64)
    e, f = torch.floor(n / 8), n % 8
    return torch.where(e == 0, f * 2.0 ** -9, (8 + f) * torch.exp2(e - 10))


def _near64(v):
    grid = _grid64(v.device)
    middle = (grid[1:] + grid[:-1]) / 2
    a = v.abs().contiguous()
    n = torch.searchsorted(middle, a)
    tie = (n < middle.numel()) & (middle[n.clamp(max=middle.numel() - 1)] == a)
    n = n + (tie & (n % 2 == 1))
    return torch.copysign(grid[n], v)


def _scale64(amax):
    return torch.maximum((amax / 448).float().double(), torch.tensor(2.0 ** -80, dtype=torch.float64, device=amax.device))


def _rows64(x):
    """x [R, C] after quantization in groups of 128 along C, as the values it stands for."""
    x = x.double()
    R, C = x.shape
    full = torch.zeros((R, _padded(C)), dtype=torch.float64, device=x.device)
    full[:, :C] = x
    g = full.view(R, -1, 128)
    s = _scale64(g.abs().max(2).values)[:, :, None]
    return (_near64(g / s) * s).view(R, -1)[:, :C]


def _blocks64(w):
    """w [M, K] after quantization in blocks of 128 x 128."""
    w = w.double()
    M, K = w.shape
    full = torch.zeros((_padded(M), _padded(K)), dtype=torch.float64, device=w.device)
    full[:M, :K] = w
    b = full.view(_padded(M) // 128, 128, _padded(K) // 128, 128).transpose(1, 2)
    s = _scale64(b.abs().flatten(2).max(2).values)[:, :, None, None]
    return (_near64(b / s) * s).transpose(1, 2).reshape(full.shape)[:M, :K]


def _given64(codes, scales, K):
    """The weights that given codes [M, padded K] and scales stand for."""
    M = codes.shape[0]
    n = (codes & 127).long()
    v = _grid64(codes.device)[n] * torch.where(codes > 127, -1.0, 1.0).double()
    r = torch.arange(M, device=codes.device) // 128
    k = torch.arange(codes.shape[1], device=codes.device) // 128
    return (v * scales.double()[r][:, k])[:, :K]


def _exact_linear(s):
    return _rows64(s["x"]) @ _given64(s["codes"], s["scales"], s["case"]["K"]).t()


def _exact_linear_train(s):
    w = _blocks64(s["w"])
    dw = _rows64(s["dy"].t()) @ _rows64(s["x"].t()).t()
    return {"y": _rows64(s["x"]) @ w.t(), "dx": _rows64(s["dy"]) @ w, "dw": dw}


def _exact_experts(s):
    c, ids = s["case"], s["ids"].flatten()
    N, S, M, K = c["N"], c["S"], c["M"], c["K"]
    rows = _rows64(s["x"].reshape(-1, K))
    of = torch.arange(N * S, device=ids.device)
    of = of if c["per_slot"] else of // S
    y = torch.zeros((N * S, M), dtype=torch.float64, device=ids.device)
    for e in range(c["E"]):
        mine = (ids == e).nonzero().flatten()
        if mine.numel():
            y[mine] = rows[of[mine]] @ _given64(s["codes"][e], s["scales"][e], K).t()
    return y.view(N, S, M)


def _exact_experts_train(s):
    c, ids, x, dout = s["case"], s["ids"].flatten(), s["x"], s["dy"]
    N, S, E, M, K = c["N"], c["S"], c["E"], c["M"], c["K"]
    token = torch.arange(N * S, device=ids.device) // S
    weights = s["weights"].double().flatten()
    dpairs = (weights[:, None] * dout.double()[token]).float().to(x.dtype)
    rows, drows = _rows64(x), _rows64(dpairs)
    y = torch.zeros((N * S, M), dtype=torch.float64, device=ids.device)
    dx = torch.zeros((N * S, K), dtype=torch.float64, device=ids.device)
    dw = torch.zeros((E, M, K), dtype=torch.float64, device=ids.device)
    for e in range(E):
        mine = (ids == e).nonzero().flatten()
        if mine.numel():
            w = _blocks64(s["w"][e])
            y[mine] = rows[token[mine]] @ w.t()
            dx[mine] = drows[mine] @ w
            dw[e] = _rows64(dpairs[mine].t()) @ _rows64(x[token[mine]].t()).t()
    return {"out": (weights[:, None] * y).view(N, S, M).sum(1), "dx": dx.view(N, S, K).sum(1), "dw": dw,
            "dweights": (y * dout.double()[token]).sum(1).view(N, S)}


def _exact_route(s):
    c, l = s["case"], s["logits"].double()
    N, E, S = c["N"], c["E"], c["S"]
    index = torch.arange(E, device=l.device)
    rank = torch.zeros((N, E), dtype=torch.int64, device=l.device)
    for j in range(E):
        rank += (l[:, j:j + 1] > l) | ((l[:, j:j + 1] == l) & (index > j))
    here = (rank < S) & (l > -math.inf)
    alive = here.any(1)
    p = torch.zeros_like(l)
    p[alive] = torch.softmax(l[alive], 1)
    tokens = int(alive.sum())
    counts = here.sum(0)
    kept = p * here
    total = torch.where(alive, kept.sum(1), torch.ones_like(kept[:, 0]))[:, None] if c["normalise"] else torch.ones_like(p[:, :1])
    order = torch.argsort(rank, 1)[:, :S]
    some = here.gather(1, order)
    weights = torch.where(some, kept.gather(1, order) / total, 0.0)
    f = counts.double() * E / (S * max(tokens, 1))
    got = {"ids": torch.where(some, order, -1).to(torch.int32), "weights": weights,
           "counts": torch.cat([counts, alive.sum()[None]]).to(torch.int32),
           "loss": BALANCE_COEF * (f * p.sum(0)).sum() / max(tokens, 1)}
    if c["train"]:
        dw = torch.where(some, s["dweights"].double(), 0.0)
        if c["normalise"]:
            dw = torch.where(some, dw - (dw * weights).sum(1, keepdim=True), 0.0) / total
        dp = s["dloss"].double() * BALANCE_COEF / max(tokens, 1) * f.repeat(N, 1)
        dp.scatter_add_(1, order, dw)
        got["dlogits"] = p * dp - p * (p * dp).sum(1, keepdim=True)
    return got


def exact(case, seed):
    s = _inputs(case, seed)
    return {"linear": _exact_linear, "linear_train": _exact_linear_train, "experts": _exact_experts,
            "experts_train": _exact_experts_train, "route": _exact_route}[case["kind"]](s)
