"""Measured cases of what a served decoder layer does between its projections: norms and rotation of the heads, the paged
key-value cache, and attention over it and over whole prompts.

Kinds of case (sizes: the heads of the decode-layer projections of qmm_synth.workloads, 32 query and 8 key heads of 128 and
16 and 8 of them, and generic odd ones):

``rope``    queries and keys of T tokens: each head divided by its root mean square, times a weight, then rotated by the
            token's position.
``step``    the same for a decode step's tokens, the keys and values written to their slots of a paged cache as well.
``cache``   new tokens' keys and values written to a paged cache, then the sequences read back, packed one after another:
            what a prompt that arrives in parts does before its attention.
``attend``  one new token per sequence over the tokens that a paged cache holds of it.
``prompt``  causal attention of packed sequences; with a prefix the keys are longer than the queries and end with them.

An 8-bit cache holds e4m3 codes and one fp32 scale per token and head; ``cache`` returns the values they stand for.
"""

import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6
BASE = 1.0e6  # of the rotation's frequencies
E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -80


# ---- cases -------------------------------------------------------------------------------------

def listed():
    return [
        # the query and key heads of an 8192-token prefill, slices of one buffer of all three projections
        dict(name="rope_prompt_8192", kind="rope", T=8192, Hq=32, H=8, D=128, R=128, x="bf16", dtype="bf16",
             interleaved=False, fused=True, far=131072),
        # the fp32 outputs of the block-format projections, odd head counts, part of a head rotated in neighbouring pairs
        dict(name="rope_odd_333", kind="rope", T=333, Hq=15, H=5, D=96, R=64, x="f32", dtype="f16", interleaved=True,
             fused=False, far=1000000),
        # one decode step of 16 sequences
        dict(name="step_16", kind="step", B=16, length=512, page=64, Hq=32, H=8, D=128, R=128, x="f32", dtype="f16"),
        # a 2048-token part of four prompts joins what an 8-bit cache already holds of them
        dict(name="cache_e4m3_16384", kind="cache", B=4, T=2048, length=16384, page=64, H=8, D=128, x="bf16",
             cache="e4m3", dtype="bf16"),
        # three sequences get five tokens between them
        dict(name="cache_e4m3_odd", kind="cache", B=3, T=5, length=333, page=16, H=3, D=80, x="f32", cache="e4m3",
             dtype="f16"),
        # one short sequence: latency
        dict(name="attend_1", kind="attend", B=1, length=777, page=64, Hq=16, H=8, D=128, cache="f16", dtype="f16"),
        # a batch of sequences of many lengths
        dict(name="attend_batch_64", kind="attend", B=64, length=8192, page=64, Hq=32, H=8, D=128, cache="bf16",
             dtype="bf16"),
        # two long documents in an 8-bit cache
        dict(name="attend_e4m3_long", kind="attend", B=2, length=131072, page=128, Hq=32, H=8, D=128, cache="e4m3",
             dtype="bf16"),
        # heads and head lengths that fill no tile, small pages
        dict(name="attend_odd_13", kind="attend", B=13, length=1500, page=16, Hq=21, H=3, D=80, cache="bf16",
             dtype="bf16"),
        # a few short prompts
        dict(name="prompt_short_5", kind="prompt", B=5, length=40, prefix=0, Hq=16, H=8, D=128, dtype="f16"),
        # prompts of many lengths, parts of which the cache held before
        dict(name="prompt_packed_16", kind="prompt", B=16, length=1024, prefix=1024, Hq=32, H=8, D=128, dtype="bf16"),
        # one long prompt
        dict(name="prompt_long_8192", kind="prompt", B=1, length=8192, prefix=0, Hq=32, H=8, D=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "step", "cache", "attend", "attend", "prompt", "prompt"])
    D = rng.choice([32, 64, 80, 96, 112, 128, 128, 256])
    H = rng.choice([1, 2, 3, 4, 5, 8])
    case = dict(kind=kind, H=H, D=D)
    sixteen = rng.choice(["f16", "bf16"])
    page = rng.choice([16, 32, 64, 128, 256])
    if kind in ("rope", "step"):
        R = rng.choice([16, 32, D // 32 * 16, D, D])
        case.update(Hq=H * rng.randint(1, 8), R=min(R, D), x=rng.choice(sorted(DTYPES)))
        if kind == "step":
            case.update(B=_log(rng, 1, 256), length=_log(rng, 1, 512), page=page, dtype=sixteen)
        else:
            case.update(T=_log(rng, 1, 8192), dtype=rng.choice([case["x"], sixteen]), interleaved=rng.random() < 0.5,
                        fused=rng.random() < 0.5, far=_log(rng, 8192, 1000000))
    elif kind == "cache":
        B = _log(rng, 1, 32)
        length = _log(rng, 1, 16384)
        case.update(B=B, length=max(1, min(length, 65536 // B)), page=page, x=rng.choice(sorted(DTYPES)),
                    cache=rng.choice(["e4m3", "e4m3", sixteen]), dtype=sixteen)
        case["T"] = _log(rng, 1, max(1, case["length"] * B // 4))
    elif kind == "attend":
        B = _log(rng, 1, 128)
        cache = rng.choice([sixteen, "e4m3"])
        most = int(1.0e9 / (B * H * D * 4))
        case.update(B=B, length=min(_log(rng, 1, 131072), most), page=page, Hq=H * rng.randint(1, 16), cache=cache,
                    dtype=sixteen)
    else:
        B = _log(rng, 1, 32)
        case.update(B=B, Hq=H * rng.randint(1, 8), dtype=sixteen)
        length, prefix = _log(rng, 1, 8192), rng.choice([0, 0, _log(rng, 1, 4096)])
        while B * case["Hq"] * D * length * (length + prefix) > 1.2e11 or B * length * case["Hq"] * D > 1e8:
            length = length * 3 // 4
        case.update(length=max(1, length), prefix=prefix)
    return case


def _lengths(case, key, most, least=0.25):
    """Lengths of the sequences: the first is the longest, the others between a quarter of it and all of it."""
    rng = random.Random("%s %d %d %d" % (key, case["B"], most, case["D"]))
    return [most] + [max(1, int(most * rng.uniform(least, 1.0))) for _ in range(case["B"] - 1)]


def _new_tokens(case):
    """Of a `cache` case: lengths after the write, and how many of each sequence's tokens are new."""
    lengths = _lengths(case, "cache", case["length"])
    B, T = case["B"], case["T"]
    new = [min(n, T // B + (1 if b < T % B else 0)) for b, n in enumerate(lengths)]
    return lengths, new


def _prompt_lengths(case):
    n = _lengths(case, "prompt", case["length"], 0.05)
    before = _lengths(case, "prefix", case["prefix"], 0.0) if case["prefix"] else [0] * case["B"]
    return n, [a + b for a, b in zip(n, before)]


def work(case):
    kind, H, D = case["kind"], case["H"], case["D"]
    if kind in ("rope", "step"):
        T = case.get("T", case.get("B"))
        i, o = DTYPES[case["x"]].itemsize, DTYPES[case["dtype"]].itemsize
        heads = case["Hq"] + H + (H if kind == "step" else 0)
        return {"bytes": float(T * heads * D * (i + o) + 4 * T * (2 if kind == "step" else 1) + 4 * case["R"] // 2 + 8 * D),
                "flops": float(T * heads * D * 8)}
    if kind == "cache":
        lengths, new = _new_tokens(case)
        i, o = DTYPES[case["x"]].itemsize, DTYPES[case["dtype"]].itemsize
        row = D + 4 if case["cache"] == "e4m3" else 2 * D
        return {"bytes": float(2 * H * (sum(new) * (D * i + row) + sum(lengths) * (row + D * o))),
                "flops": float(2 * H * D * (3 * sum(new) + sum(lengths)))}
    if kind == "attend":
        tokens = sum(_lengths(case, "attend", case["length"]))
        row = D + 4 if case["cache"] == "e4m3" else 2 * D
        return {"bytes": float(2 * tokens * H * row + 4 * case["B"] * case["Hq"] * D), "flops": 4.0 * case["Hq"] * D * tokens}
    n, m = _prompt_lengths(case)
    pairs = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(n, m))
    return {"bytes": float(4 * sum(n) * case["Hq"] * D + 4 * sum(m) * H * D), "flops": 4.0 * case["Hq"] * D * pairs}


# ---- inputs ------------------------------------------------------------------------------------

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _keys(g, T, H, D):
    """Keys have channels that are large for every token."""
    return _randn(g, T, H, D) + _randn(g, 1, H, D) * (torch.rand((1, H, D), generator=g, device="cuda") < 0.06) * 4.0


def _starts(lengths):
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return out


def _table(g, lengths, page):
    """Pages of the sequences in any order; entries past a sequence's last page name none."""
    need = [-(-n // page) for n in lengths]
    order = torch.randperm(sum(need), generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lengths), max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, sum(need)


def _slots(table, page, b, first, count):
    t = torch.arange(first, first + count, device="cuda")
    return (table[b, t // page].long() * page + t % page).to(torch.int32)


def _frequencies(R):
    return (BASE ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)).float()


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    kind, H, D = case["kind"], case["H"], case["D"]
    s = dict(case=dict(case))
    if kind in ("rope", "step"):
        T, Hq, dtype = case.get("T", case.get("B")), case["Hq"], DTYPES[case["x"]]
        if case.get("fused") or kind == "step":
            rows = (_randn(g, T, Hq + 2 * H, D) * 2.0).to(dtype)
            s["q"], s["k"], s["v"] = rows[:, :Hq], rows[:, Hq:Hq + H], rows[:, Hq + H:]
        else:
            s["q"], s["k"] = (_randn(g, T, Hq, D) * 2.0).to(dtype), (_randn(g, T, H, D) * 2.0).to(dtype)
        s["q_weight"], s["k_weight"] = 1.0 + 0.2 * _randn(g, D), 1.0 + 0.2 * _randn(g, D)
        s["inv_freq"] = _frequencies(case["R"])
    if kind == "rope":
        s["positions"] = torch.randint(0, case["far"], (T,), generator=g, device="cuda", dtype=torch.int32)
    elif kind == "step":
        lengths = _lengths(case, "step", case["length"])
        table, pages = _table(g, lengths, case["page"])
        s["positions"] = torch.tensor([n - 1 for n in lengths], dtype=torch.int32, device="cuda")
        s["slots"] = torch.cat([_slots(table, case["page"], b, n - 1, 1) for b, n in enumerate(lengths)])
        for x in "kv":
            s["cache_" + x] = _randn(g, pages, H, case["page"], D).to(DTYPES[case["dtype"]])
    elif kind == "cache":
        lengths, new = _new_tokens(case)
        table, pages = _table(g, lengths, case["page"])
        s["table"], s["starts"] = table, torch.tensor(_starts(lengths), dtype=torch.int32, device="cuda")
        s["total"] = sum(lengths)
        s["slots"] = torch.cat([_slots(table, case["page"], b, n - a, a) for b, (n, a) in enumerate(zip(lengths, new))])
        s["k"], s["v"] = (f(g, sum(new), H, D).to(DTYPES[case["x"]]) for f in (_keys, _randn))
        _held(s, g, pages)
    elif kind == "attend":
        lengths = _lengths(case, "attend", case["length"])
        s["table"], pages = _table(g, lengths, case["page"])
        s["lengths"], s["longest"] = torch.tensor(lengths, dtype=torch.int32, device="cuda"), max(lengths)
        s["q"] = (_randn(g, case["B"], case["Hq"], D) * 1.5).to(DTYPES[case["dtype"]])
        _held(s, g, pages)
    else:
        n, m = _prompt_lengths(case)
        dtype, Hq = DTYPES[case["dtype"]], case["Hq"]
        s["n"], s["m"] = n, m
        s["starts"] = torch.tensor(_starts(n), dtype=torch.int32, device="cuda")
        if case["prefix"]:
            s["k_starts"] = torch.tensor(_starts(m), dtype=torch.int32, device="cuda")
            s["q"] = (_randn(g, sum(n), Hq, D) * 1.5).to(dtype)
            s["k"], s["v"] = _keys(g, sum(m), H, D).to(dtype), _randn(g, sum(m), H, D).to(dtype)
        else:
            s["k_starts"] = s["starts"]
            rows = torch.cat([_randn(g, sum(n), Hq, D) * 1.5, _keys(g, sum(n), H, D), _randn(g, sum(n), H, D)], 1).to(dtype)
            s["q"], s["k"], s["v"] = rows[:, :Hq], rows[:, Hq:Hq + H], rows[:, Hq + H:]
    return s


def _held(s, g, pages):
    """What the cache holds before the call, in every slot of its pages."""
    c = s["case"]
    H, D, page = c["H"], c["D"], c["page"]
    for name, f in (("k", _keys), ("v", _randn)):
        if c["cache"] == "e4m3":
            codes = torch.empty((pages, H, page, D), dtype=torch.uint8, device="cuda")
            scales = torch.empty((pages, H, page), device="cuda")
            step = max(1, (1 << 22) // (H * page * D) * page)  # tokens at a time: quantized in 64 bits
            for p in range(0, pages, max(1, step // page)):
                some = min(max(1, step // page), pages - p)
                x = f(g, some * page, H, D).view(some, page, H, D).transpose(1, 2)
                values, scale = _quantize(x)
                codes[p:p + some] = values.to(torch.float8_e4m3fn).view(torch.uint8)
                scales[p:p + some] = scale
            s["cache_" + name], s["scales_" + name] = codes, scales
        else:
            held = torch.empty((pages, H, page, D), dtype=DTYPES[c["cache"]], device="cuda")
            for p in range(0, pages, 64):
                some = min(64, pages - p)
                held[p:p + some] = f(g, some * page, H, D).view(some, page, H, D).transpose(1, 2)
            s["cache_" + name] = held


def prepare(case, seed):
    s = _inputs(case, seed)
    if own and "cache_k" in s:
        import block_quantized_weight_matmul_amd as q
        s["cache"] = q.KVCache(s["cache_k"], s["cache_v"], s.get("scales_k"), s.get("scales_v"))
    return s


# ---- the plain forms ---------------------------------------------------------------------------

def _e4m3(v):
    """Nearest e4m3 value (ties to even) of the float64 v, |v| <= 448."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(e - 1, min=-6) - 3)
    return torch.round(v / step) * step


def _quantize(x):
    """One scale per row of the last axis: e4m3 values and scales, both fp32."""
    x = x.float()
    s = torch.clamp((x.abs().amax(-1).double() / E4M3_MAX).float(), min=MIN_SCALE)
    return _e4m3(x.double() / s.double().unsqueeze(-1)).float(), s


def _norm(x, weight):
    x = x.float()
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * weight


def _rotate(x, positions, inv_freq, interleaved):
    angle = positions.double()[:, None, None] * inv_freq.double()  # far positions lose theirs in 32 bits
    c, s = torch.cos(angle).float(), torch.sin(angle).float()
    R = 2 * inv_freq.shape[0]
    r, rest = x[..., :R], x[..., R:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = r[..., :R // 2], r[..., R // 2:]
        r = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([r, rest], -1)


def _plain_heads(s):
    c = s["case"]
    inter = c.get("interleaved", False)
    return tuple(_rotate(_norm(s[x], s[x + "_weight"]), s["positions"], s["inv_freq"], inter).to(DTYPES[c["dtype"]])
                 for x in "qk")


def _plain_step(s):
    q, k = _plain_heads(s)
    page, slots = s["case"]["page"], s["slots"].long()
    at, row = slots // page, slots % page
    s["cache_k"][at, :, row] = k
    s["cache_v"][at, :, row] = s["v"].to(k.dtype)
    return {"q": q, "k": s["cache_k"], "v": s["cache_v"]}


def _values(s, x):
    """The cache as the values it stands for, fp32."""
    if s["case"]["cache"] == "e4m3":
        return s["cache_" + x].view(torch.float8_e4m3fn).float() * s["scales_" + x].unsqueeze(-1)
    return s["cache_" + x].float()


def _plain_cache(s):
    c = s["case"]
    page, slots, out = c["page"], s["slots"].long(), {}
    at, row = slots // page, slots % page
    owner = torch.searchsorted(s["starts"][1:].long(), torch.arange(s["total"], device="cuda"), right=True)
    t = torch.arange(s["total"], device="cuda") - s["starts"].long()[owner]
    pages = s["table"].long()[owner, t // page]
    for x in "kv":
        if c["cache"] == "e4m3":
            values, scales = _quantize(s[x])
            s["cache_" + x][at, :, row] = values.to(torch.float8_e4m3fn).view(torch.uint8)
            s["scales_" + x][at, :, row] = scales
            codes = s["cache_" + x][pages, :, t % page]
            got = codes.view(torch.float8_e4m3fn).float() * s["scales_" + x][pages, :, t % page].unsqueeze(-1)
        else:
            s["cache_" + x][at, :, row] = s[x].to(s["cache_" + x].dtype)
            got = s["cache_" + x][pages, :, t % page].float()
        out[x] = got.to(DTYPES[c["dtype"]])
    return out


def _softmax(scores, visible):
    """Softmax over the last axis of what is visible; a row that sees nothing is zeros."""
    scores = torch.where(visible, scores, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - torch.where(top > float("-inf"), top, 0.0))
    return e / torch.where(top > float("-inf"), e.sum(-1, keepdim=True), 1.0)


def _plain_attend(s):
    c, q, table = s["case"], s["q"], s["table"]
    B, Hq, D = q.shape
    H, page = c["H"], c["page"]
    pages = table.clamp(min=0).long()
    L = pages.shape[1] * page
    seen = torch.arange(L, device="cuda")[None] < s["lengths"][:, None]

    def rows(x):  # [B, H, L, D]
        r = s["cache_" + x][pages].transpose(1, 2).reshape(B, H, L, D)
        if c["cache"] == "e4m3":
            return r.view(torch.float8_e4m3fn).float() * s["scales_" + x][pages].transpose(1, 2).reshape(B, H, L, 1)
        return r.float()

    scores = torch.matmul(q.float().view(B, H, Hq // H, D), rows("k").transpose(2, 3).contiguous()) / math.sqrt(D)
    p = _softmax(scores, seen[:, None, None])
    return torch.matmul(p, rows("v")).view(B, Hq, D).to(q.dtype)


def _plain_prompt(s):
    q, k, v = s["q"], s["k"], s["v"]
    G, out = q.shape[1] // k.shape[1], []
    qs, ks = _starts(s["n"]), _starts(s["m"])
    for b, (n, m) in enumerate(zip(s["n"], s["m"])):
        qb = q[qs[b]:qs[b + 1]].float().transpose(0, 1)
        kb = k[ks[b]:ks[b + 1]].float().repeat_interleave(G, 1).permute(1, 2, 0).contiguous()
        vb = v[ks[b]:ks[b + 1]].float().repeat_interleave(G, 1).transpose(0, 1).contiguous()
        scores = torch.matmul(qb.contiguous(), kb) / math.sqrt(q.shape[2])
        seen = torch.arange(m, device="cuda")[None] <= torch.arange(n, device="cuda")[:, None] + (m - n)
        out.append(torch.matmul(_softmax(scores, seen[None]), vb).transpose(0, 1))
    return torch.cat(out).to(q.dtype)


# ---- the library's calls -----------------------------------------------------------------------

def _own_rope(s):
    import block_quantized_weight_matmul_amd as q
    c = s["case"]
    return q.head_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], s["q_weight"], s["k_weight"], eps=EPS,
                            interleaved=c["interleaved"], dtype=DTYPES[c["dtype"]])


def _own_step(s):
    q = s["cache"].norm_rope_write(s["q"], s["k"], s["v"], s["slots"], s["positions"], s["inv_freq"], s["q_weight"],
                                   s["k_weight"], eps=EPS)
    return {"q": q, "k": s["cache_k"], "v": s["cache_v"]}


def _own_cache(s):
    s["cache"].write(s["k"], s["v"], s["slots"])
    k, v = s["cache"].read(s["table"], s["starts"], s["total"], dtype=DTYPES[s["case"]["dtype"]])
    return {"k": k, "v": v}


def _own_attend(s):
    return s["cache"].attend(s["q"], s["table"], s["lengths"], max_length=s["longest"])


def _own_prompt(s):
    import block_quantized_weight_matmul_amd as q
    return q.attend_prompt(s["q"], s["k"], s["v"], s["starts"], s["k_starts"])


def run(state):
    kind = state["case"]["kind"]
    if own:
        return {"rope": _own_rope, "step": _own_step, "cache": _own_cache, "attend": _own_attend,
                "prompt": _own_prompt}[kind](state)
    return {"rope": _plain_heads, "step": _plain_step, "cache": _plain_cache, "attend": _plain_attend,
            "prompt": _plain_prompt}[kind](state)


# ---- the definitions in 64 bits ----------------------------------------------------------------
# Scales of a cache are fp32 numbers and its codes e4m3 ones in the definition too.

def _heads64(x, weight, positions, inv_freq, interleaved):
    x = x.double()
    D, half = x.shape[-1], inv_freq.shape[0]
    y = x * (x.pow(2).sum(-1, keepdim=True) / D + EPS).pow(-0.5) * weight.double()
    first = torch.arange(half, device=x.device) * (2 if interleaved else 1)
    second = first + (1 if interleaved else half)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                       positions.double().view(-1, 1, 1) * inv_freq.double())
    z = torch.complex(y[..., first], y[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_rope(s):
    c = s["case"]
    inter = c.get("interleaved", False)
    return tuple(_heads64(s[x], s[x + "_weight"], s["positions"], s["inv_freq"], inter) for x in "qk")


def _exact_step(s):
    q, k = _exact_rope(s)
    got = {"q": q, "k": s["cache_k"].double(), "v": s["cache_v"].double()}
    for t, slot in enumerate(s["slots"].tolist()):
        page, row = divmod(slot, s["case"]["page"])
        got["k"][page, :, row], got["v"][page, :, row] = k[t], s["v"][t].double()
    return got


def _near64(x):
    """Rows of x as e4m3 codes times a scale stand for them."""
    n = torch.arange(127, device=x.device, dtype=torch.float64)
    grid = torch.where(n < 8, n * 2.0 ** -9, (8 + n % 8) * torch.exp2(torch.floor(n / 8) - 10))
    middle = (grid[1:] + grid[:-1]) / 2
    s = (x.abs().max(-1, keepdim=True).values / 448).float().double().clamp(min=2.0 ** -80)
    a = (x / s).abs().contiguous()
    at = torch.searchsorted(middle, a)
    tie = (at < 126) & (middle[at.clamp(max=125)] == a) & (at % 2 == 1)
    return torch.copysign(grid[at + tie], x) * s


def _stored64(s, x):
    """The cache's values, [pages, H, page, D]."""
    if s["case"]["cache"] == "e4m3":
        return s["cache_" + x].view(torch.float8_e4m3fn).double() * s["scales_" + x].double()[..., None]
    return s["cache_" + x].double()


def _exact_cache(s):
    c, out = s["case"], {}
    page, H, D = c["page"], c["H"], c["D"]
    lengths = _new_tokens(c)[0]
    for x in "kv":
        flat = _stored64(s, x).transpose(1, 2).reshape(-1, H, D)  # by slot
        new = s[x].double()
        flat[s["slots"].long()] = _near64(new) if c["cache"] == "e4m3" else new
        parts = [flat[_slots(s["table"], page, b, 0, n).long()] for b, n in enumerate(lengths)]
        out[x] = torch.cat(parts)
    return out


def _exact_attend(s):
    c, q = s["case"], s["q"].double()
    H, D, page = c["H"], c["D"], c["page"]
    out = torch.zeros_like(q)
    for b, n in enumerate(_lengths(c, "attend", c["length"])):
        pages = s["table"][b, :-(-n // page)].long()
        part = {"case": c}
        for x in "kv":
            part["cache_" + x] = s["cache_" + x][pages]
            if c["cache"] == "e4m3":
                part["scales_" + x] = s["scales_" + x][pages]
        k, v = (_stored64(part, x).transpose(0, 1).reshape(H, -1, D)[:, :n] for x in "kv")
        for h in range(q.shape[1]):
            a = k[h * H // q.shape[1]] @ q[b, h] * D ** -0.5
            out[b, h] = torch.softmax(a, 0) @ v[h * H // q.shape[1]]
    return out


def _exact_prompt(s):
    q, k, v = s["q"], s["k"], s["v"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    Hq, H, D = q.shape[1], k.shape[1], q.shape[2]
    at = kat = 0
    for n, m in zip(s["n"], s["m"]):
        for h in range(Hq):
            kb, vb = k[kat:kat + m, h * H // Hq].double(), v[kat:kat + m, h * H // Hq].double()
            a = (q[at:at + n, h].double() @ kb.t()) * D ** -0.5
            a += torch.full_like(a, -math.inf).triu(m - n + 1)
            out[at:at + n, h] = torch.softmax(a, 1) @ vb
        at, kat = at + n, kat + m
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    return {"rope": _exact_rope, "step": _exact_step, "cache": _exact_cache, "attend": _exact_attend,
            "prompt": _exact_prompt}[case["kind"]](s)
