"""The 4-bit (MXFP4) and expert operators: cases, plain forms and the library's calls.

MXFP4: e2m1 codes, two to a byte (the even column in the low nibble), and one power-of-two scale byte (2^(b - 127))
for each 32 consecutive columns of a row. A case is a dict of plain values. `prepare` makes what a program holds
before the call, `run` makes one pass: in elementary torch operations where `own` is false, through
dense_fp8_gemm_b200.spense where it is true. `exact` computes the same from the definitions in 64 bits.
"""
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # The hidden state of one decoded token, quantised ahead of its projections: a call that is all latency.
        {"name": "quantize one token", "op": "quantize", "tokens": 1, "rows": 0, "spare": 0, "K": 5120, "dtype": "bf16"},
        # A long prompt's hidden states, each copied to its four experts while it is quantised; the batch is padded.
        {"name": "quantize routed prompt", "op": "quantize", "tokens": 8192, "rows": 32768, "spare": 77, "K": 5120,
         "dtype": "bf16"},
        # q, k and v of one token: 28 MB of weights, about as short as a product of this library gets.
        {"name": "gemm qkv 1 token", "op": "gemm", "M": 1, "N": 10240, "K": 5120},
        # The down projection for a decoding batch of odd size: 40 tiles of weight rows, a long contraction.
        {"name": "gemm down 45 tokens", "op": "gemm", "M": 45, "N": 5120, "K": 27648},
        # gate and up over a whole prompt: bound by the tensor cores.
        {"name": "gemm gate+up 8192 tokens", "op": "gemm", "M": 8192, "N": 51200, "K": 5120},
        # Four decoded tokens on eight experts each: every chosen expert's weights are read for one row or two.
        {"name": "experts decode", "op": "experts", "E": 64, "T": 32, "spare": 0, "N": 2560, "K": 5120, "skew": 0.3},
        # A decoding batch of 64 tokens over many experts, unevenly loaded, in a padded buffer.
        {"name": "experts batch", "op": "experts", "E": 128, "T": 509, "spare": 3, "N": 2560, "K": 2048, "skew": 0.8},
        # A long prompt over 32 experts, unevenly loaded: large ragged products.
        {"name": "experts prompt", "op": "experts", "E": 32, "T": 32768, "spare": 300, "N": 5120, "K": 2560,
         "skew": 0.6},
        # The router's choice for a small decoding batch, as top-k gives it.
        {"name": "sort decode", "op": "sort", "M": 16, "k": 8, "E": 128, "ids": "i64", "drop": 0.0},
        # A long prompt's choices, some of them another device's experts.
        {"name": "sort prompt", "op": "sort", "M": 16384, "k": 8, "E": 256, "ids": "i32", "drop": 0.1},
        # The weighted sum of the experts' rows for a small decoding batch.
        {"name": "combine decode", "op": "combine", "M": 16, "k": 8, "N": 5120, "drop": 0.0},
        # The same for a prompt of odd length with dropped choices.
        {"name": "combine prompt", "op": "combine", "M": 8191, "k": 8, "N": 5120, "drop": 0.1},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "experts", "experts", "sort", "combine"])
    if op == "quantize":
        tokens, K = _log(rng, 1, 16384), 32 * _log(rng, 1, 864)
        rows = rng.choice([0, 1, 1])
        rows = rows and max(1, min(32768, int(tokens * rng.uniform(0.3, 8.0))))
        return {"op": op, "tokens": tokens, "rows": rows, "spare": rng.choice([0, 5, 130]) if rows else 0, "K": K,
                "dtype": rng.choice(["bf16", "bf16", "f16", "f32"])}
    if op == "gemm":
        M, N, K = _log(rng, 1, 8192), _log(rng, 65, 55296), 32 * _log(rng, 4, 864)
        N = N if rng.random() < 0.3 else -(-N // 8) * 8
        while M * N * K > 8192 * 51200 * 5120:
            M = M // 2 + 1
        return {"op": op, "M": M, "N": N, "K": K}
    if op == "experts":
        E, T, N, K = _log(rng, 2, 128), _log(rng, 1, 32768), 8 * _log(rng, 16, 640), 32 * _log(rng, 8, 160)
        while E * N * K > 128 * 2560 * 5120:
            E = E // 2 + 1
        return {"op": op, "E": E, "T": T, "spare": rng.choice([0, 0, 1, 200]), "N": N, "K": K,
                "skew": round(rng.uniform(0.0, 1.2), 2)}
    if op == "sort":
        return {"op": op, "M": _log(rng, 1, 32768), "k": rng.randint(1, 8), "E": _log(rng, 8, 512),
                "ids": rng.choice(["i32", "i64"]), "drop": rng.choice([0.0, 0.1, 0.9])}
    return {"op": op, "M": _log(rng, 1, 16384), "k": rng.randint(1, 8), "N": _log(rng, 64, 8192),
            "drop": rng.choice([0.0, 0.1, 0.9])}


def _counts(case):
    """Rows of each expert, largest first: T split in proportion to (i + 1)^-skew."""
    p = [(i + 1.0) ** -case["skew"] for i in range(case["E"])]
    c = [int(case["T"] * x / sum(p)) for x in p]
    left = case["T"] - sum(c)
    return [x + left // case["E"] + (1 if i < left % case["E"] else 0) for i, x in enumerate(c)]


def _activations(rows, K, gen, dtype=torch.float32):
    """Hidden states: normal, each token with its own size, and some channels that are much larger in every token."""
    x = torch.randn(rows, K, device="cuda", generator=gen)
    x *= torch.exp(0.3 * torch.randn(rows, 1, device="cuda", generator=gen))
    x *= torch.where(torch.rand(K, device="cuda", generator=gen) < 0.01, 12.0, 1.0)
    return x.to(dtype)


def _weights(count, N, K, gen):
    """Codes [count, N, K / 2] and scale bytes [count, N, K / 32] of weights drawn from N(0, 0.02)."""
    wq = torch.empty(count, N, K // 2, dtype=torch.uint8, device="cuda")
    ws = torch.empty(count, N, K // 32, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (N * K))
    for i in range(0, count, step):
        n = min(step, count - i)
        q, s = _quantize(0.02 * torch.randn(n * N, K, device="cuda", generator=gen))
        wq[i:i + n], ws[i:i + n] = q.view(n, N, K // 2), s.view(n, N, K // 32)
    return wq, ws


def _quantize(x):
    """MXFP4 of float32 rows: codes [rows, K / 2], scale bytes [rows, K / 32]. A block's exponent is that of its largest
    magnitude less 2 (the exponent of 6, the largest code), a code the nearest level, ties to the even one."""
    rows, K = x.shape
    b = x.view(rows, K // 32, 32)
    amax = b.abs().amax(dim=2)
    e = (torch.frexp(amax).exponent - 3).clamp(-127, 127)
    e = torch.where(amax == 0, -127, e)
    a = b.abs() * ((127 - e) << 23).to(torch.int32).view(torch.float32).unsqueeze(2)
    code = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    code = (code + 8 * torch.signbit(b).to(torch.uint8)).view(rows, K // 2, 2)
    return code[:, :, 0] + 16 * code[:, :, 1], (e + 127).to(torch.uint8)


def _words(scale):
    """Scale bytes [rows, K / 32] as words of four, column group by column group: [ceil(K / 128), rows, 4]."""
    rows, n = scale.shape
    return torch.nn.functional.pad(scale, (0, -n % 4)).view(rows, -1, 4).permute(1, 0, 2).contiguous()


def _powers(scale, dtype):
    return ((scale.to(torch.int64) + 896) << 52).view(torch.float64).to(dtype)


def _decode(q, scale, levels, dtype=torch.float32):
    """The values [..., K] of codes [..., K / 2] and scale bytes [..., K / 32]."""
    code = torch.stack((q & 15, q >> 4), dim=-1).view(*scale.shape, 32)
    return (levels[code.to(torch.int32)].to(dtype) * _powers(scale, dtype).unsqueeze(-1)).flatten(-2)


def _row_scales(words, K):
    return words.permute(1, 0, 2).flatten(1)[:, :K // 32]


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(7919 * seed + 13)
    levels = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device="cuda")
    op, s = case["op"], {"case": case, "levels": levels}
    if op == "quantize":
        s["X"] = _activations(case["tokens"], case["K"], gen, DTYPES[case["dtype"]])
        s["rows"] = None
        total = case["tokens"]
        if case["rows"]:
            total = case["rows"] + case["spare"]
            s["rows"] = torch.full((total,), -1, dtype=torch.int32, device="cuda")
            s["rows"][:case["rows"]] = torch.randint(case["tokens"], (case["rows"],), device="cuda", generator=gen)
        s["Xq"] = torch.zeros(total, case["K"] // 2, dtype=torch.uint8, device="cuda")
        s["scale"] = torch.zeros(-(-case["K"] // 128), total, 4, dtype=torch.uint8, device="cuda")
    elif op == "gemm":
        s["wq"], s["ws"] = _weights(1, case["N"], case["K"], gen)
        s["xq"], xs = _quantize(_activations(case["M"], case["K"], gen))
        s["xs"] = _words(xs)
        s["Y"] = torch.zeros(case["M"], case["N"], dtype=torch.bfloat16, device="cuda")
    elif op == "experts":
        E, T = case["E"], case["T"]
        s["wq"], s["ws"] = _weights(E, case["N"], case["K"], gen)
        s["xq"], xs = _quantize(_activations(T + case["spare"], case["K"], gen))
        s["xs"] = _words(xs)
        counts = torch.tensor(_counts(case), device="cuda")[torch.randperm(E, device="cuda", generator=gen)]
        s["offsets"] = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).to(torch.int32)
        s["Y"] = torch.zeros(T + case["spare"], case["N"], dtype=torch.bfloat16, device="cuda")
    elif op == "sort":
        M, k, E = case["M"], case["k"], case["E"]
        score = torch.randn(M, E, device="cuda", generator=gen) + torch.randn(E, device="cuda", generator=gen)
        ids = torch.topk(score, k, dim=1).indices
        ids = torch.where(torch.rand(M, k, device="cuda", generator=gen) < case["drop"], -1, ids)
        s["ids"] = ids.to(torch.int32 if case["ids"] == "i32" else torch.int64)
    else:
        M, k, N = case["M"], case["k"], case["N"]
        s["Y"] = torch.randn(M * k, N, device="cuda", generator=gen).to(torch.bfloat16)
        pos = torch.randperm(M * k, device="cuda", generator=gen).view(M, k)
        s["pos"] = torch.where(torch.rand(M, k, device="cuda", generator=gen) < case["drop"], -1, pos).to(torch.int32)
        s["weights"] = torch.softmax(torch.randn(M, k, device="cuda", generator=gen), dim=1)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own and case["op"] in ("gemm", "experts"):
        from dense_fp8_gemm_b200 import spense
        s["packed"] = spense.mx4_pack(s.pop("wq"), s.pop("ws"))
        rows = s["xq"].shape[0]
        s["call"] = spense.PreparedMx4Gemm(s["packed"], s["xq"], s["xs"], s["Y"],
                                           spense.new_workspace(spense.mx4_workspace_size(s["packed"], rows)),
                                           offsets=s.get("offsets"))
    return s


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    from dense_fp8_gemm_b200 import spense
    op = s["case"]["op"]
    if op == "quantize":
        q, scale = spense.mx4_quantize(s["X"], rows=s["rows"], Xq=s["Xq"], x_scale=s["scale"])
        return spense.mx4_dequantize(q, scale)
    if op in ("gemm", "experts"):
        s["call"]()
        return s["Y"]
    if op == "sort":
        return spense.expert_sort(s["ids"], s["case"]["E"])
    return spense.expert_combine(s["Y"], s["pos"], s["weights"])


def _run_plain(s):
    case = s["case"]
    op, levels = case["op"], s["levels"]
    if op == "quantize":
        x = s["X"]
        if s["rows"] is not None:
            x = torch.where((s["rows"] >= 0).unsqueeze(1), x[s["rows"].clamp(min=0)], 0)
        return _decode(*_quantize(x.to(torch.float32)), levels).to(torch.bfloat16)
    if op == "gemm":
        x = _decode(s["xq"], _row_scales(s["xs"], case["K"]), levels)
        return (x @ _decode(s["wq"][0], s["ws"][0], levels).t()).to(torch.bfloat16)
    if op == "experts":
        # Every expert's rows at the front of a slab of their own, one batched product, and the rows back in place.
        off, x = s["offsets"].to(torch.int64), _decode(s["xq"], _row_scales(s["xs"], case["K"]), levels)
        most = max(_counts(case))
        at = off[:-1, None] + torch.arange(most, device=off.device)
        there = at < off[1:, None]
        slab = x[torch.where(there, at, 0)]
        y = torch.bmm(slab, _decode(s["wq"], s["ws"], levels).transpose(1, 2)).to(torch.bfloat16)
        out = s["Y"].clone()
        out[at[there]] = y[there]
        return out
    if op == "sort":
        ids, E, k = s["ids"].reshape(-1).to(torch.int64), case["E"], case["k"]
        key = torch.where((ids >= 0) & (ids < E), ids, E)
        sorted_key, order = torch.sort(key, stable=True)
        offsets = torch.searchsorted(sorted_key, torch.arange(E + 1, device=key.device))
        rows = torch.where(sorted_key < E, order // k, -1)
        pos = torch.empty_like(order)
        pos[order] = torch.arange(order.numel(), device=order.device)
        pos = torch.where(key < E, pos, -1).view(-1, k)
        return offsets.to(torch.int32), rows.to(torch.int32), pos.to(torch.int32)
    pos, live = s["pos"].clamp(min=0), s["pos"] >= 0
    y = s["Y"][pos].to(torch.float32) * s["weights"].unsqueeze(2)
    return torch.where(live.unsqueeze(2), y, 0.0).sum(dim=1).to(torch.bfloat16)


def work(case):
    op = case["op"]
    if op == "quantize":
        K, total = case["K"], case["rows"] or case["tokens"]
        read = min(total, case["tokens"]) * K * (4 if case["dtype"] == "f32" else 2) + 4 * case["rows"]
        return {"bytes": read + total * (K // 2 + K // 32 + 2 * K), "flops": total * K}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * (K // 2 + K // 32) + 2 * M * N, "flops": 2 * M * N * K}
    if op == "experts":
        N, K, T = case["N"], case["K"], case["T"]
        active = sum(1 for c in _counts(case) if c)
        return {"bytes": (T + active * N) * (K // 2 + K // 32) + 2 * T * N + 4 * (case["E"] + 1),
                "flops": 2 * T * N * K}
    if op == "sort":
        n = case["M"] * case["k"]
        return {"bytes": n * (4 if case["ids"] == "i32" else 8) + 8 * n + 4 * (case["E"] + 1), "flops": 0}
    n = case["M"] * case["k"]
    live = int(n * (1 - case["drop"]))
    return {"bytes": live * 2 * case["N"] + 8 * n + 2 * case["M"] * case["N"], "flops": 2 * live * case["N"]}


def _value(q, scale):
    """Codes and row-major scale bytes as float64 values, from the formats' bit fields."""
    c = torch.stack((q.to(torch.int64) % 16, q.to(torch.int64) // 16), dim=-1).view(*scale.shape, 32)
    man, exp, neg = c % 2, c // 2 % 4, c // 8
    v = torch.where(exp == 0, 0.5 * man.double(), (1.0 + 0.5 * man.double()) * 0.5 * (1 << exp).double())
    power = torch.tensor([2.0 ** (i - 127) for i in range(256)], dtype=torch.float64, device=q.device)
    return (torch.where(neg == 1, -v, v) * power[scale.to(torch.int64)].unsqueeze(-1)).flatten(-2)


def exact(case, seed):
    op = case["op"]
    if op == "sort":
        return None
    s = _inputs(case, seed)
    if op == "quantize":
        total = s["Xq"].shape[0]
        out = torch.zeros(total, case["K"], dtype=torch.float64, device="cuda")
        levels = torch.tensor(LEVELS, dtype=torch.float64, device="cuda")
        for i in range(0, total, 4096):
            n = min(4096, total - i)
            x = s["X"][i:i + n] if s["rows"] is None else s["X"][s["rows"][i:i + n].clamp(min=0)]
            b = x.double().view(n, -1, 32)
            if s["rows"] is not None:
                b = b * (s["rows"][i:i + n] >= 0).view(n, 1, 1)
            amax = b.abs().amax(dim=2, keepdim=True)
            # amax over its fraction in [1/2, 1) is a power of two; an eighth of it is 2^(floor(log2 amax) - 2)
            unit = torch.where(amax > 0, (amax / torch.frexp(amax).mantissa / 8).clamp(min=2.0 ** -127), 1.0)
            a = (b.abs() / unit).clamp(max=6.0)
            # between the levels on both sides the nearer one, at a tie the one with an even code
            hi = torch.searchsorted(levels, a).clamp(max=7)
            lo = (hi - 1).clamp(min=0)
            up, down = levels[hi] - a, a - levels[lo]
            code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
            out[i:i + n] = (torch.sign(b) * levels[code] * unit).flatten(1)
        return out
    if op == "gemm":
        return _value(s["xq"], _row_scales(s["xs"], case["K"])) @ _value(s["wq"][0], s["ws"][0]).t()
    if op == "experts":
        x, out = _value(s["xq"], _row_scales(s["xs"], case["K"])), s["Y"].double()
        ends = s["offsets"].tolist()
        for e in range(case["E"]):
            a, b = ends[e], ends[e + 1]
            if b > a:
                out[a:b] = x[a:b] @ _value(s["wq"][e], s["ws"][e]).t()
        return out
    out = torch.zeros(case["M"], case["N"], dtype=torch.float64, device="cuda")
    for j in range(case["k"]):
        p = s["pos"][:, j]
        out += torch.where((p >= 0).unsqueeze(1), s["weights"][:, j:j + 1].double() * s["Y"][p.clamp(min=0)].double(), 0.0)
    return out
