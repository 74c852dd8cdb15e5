"""INT8 linear layers: the cases whose speed is followed, and their plain forms.

Three operators: the per-token quantizer (with the gather that dispatches tokens to experts), the
matrix product with a scale for each token and each channel, and the same product grouped by expert
with the group bounds on the device.  ``run`` computes them in elementary torch operations, or, where
``own`` is true, through the library.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one generated token's activation before a projection
        {"name": "quantize_token", "op": "quantize", "dtype": "bf16", "tokens": 1, "rows": 1, "cols": 8192, "gather": False},
        # a prefill's activation before the up-projection
        {"name": "quantize_prefill", "op": "quantize", "dtype": "bf16", "tokens": 8192, "rows": 8192, "cols": 8192,
         "gather": False},
        # a dispatch: every token goes to two experts, its row quantized into both groups
        {"name": "quantize_dispatch", "op": "quantize", "dtype": "fp16", "tokens": 4097, "rows": 8194, "cols": 4096,
         "gather": True},
        # a large weight quantized by output channel
        {"name": "quantize_weight", "op": "quantize", "dtype": "bf16", "tokens": 16384, "rows": 16384, "cols": 16384,
         "gather": False},
        # single-token generation through a large projection
        {"name": "linear_token", "op": "linear", "dtype": "bf16", "m": 1, "n": 28672, "k": 8192, "bias": False},
        # a small batch through a small projection: latency counts
        {"name": "linear_batch", "op": "linear", "dtype": "bf16", "m": 16, "n": 4096, "k": 4096, "bias": True},
        # a chunk of a ragged batch, odd in every size
        {"name": "linear_ragged", "op": "linear", "dtype": "fp16", "m": 301, "n": 5003, "k": 4099, "bias": True},
        # a chunk of prefill tokens through a square projection
        {"name": "linear_square", "op": "linear", "dtype": "bf16", "m": 4096, "n": 4096, "k": 4096, "bias": False},
        # a prefill through the up-projection of a large model
        {"name": "linear_prefill", "op": "linear", "dtype": "bf16", "m": 8192, "n": 28672, "k": 8192, "bias": False},
        # generation for eight sequences, two experts each: most of the time is the active experts' weights
        {"name": "experts_token", "op": "experts", "dtype": "bf16", "experts": 8, "rows": 16, "pad": 0, "skew": 0.0,
         "n": 14336, "k": 4096, "bias": False},
        # many small experts, a few hundred routed tokens, rows left over behind the last group
        {"name": "experts_many", "op": "experts", "dtype": "fp16", "experts": 64, "rows": 1031, "pad": 9, "skew": 3.0,
         "n": 2056, "k": 2048, "bias": True},
        # a prefill's routed tokens through eight experts' up-projection
        {"name": "experts_prefill", "op": "experts", "dtype": "bf16", "experts": 8, "rows": 8192, "pad": 0, "skew": 1.0,
         "n": 14336, "k": 4096, "bias": False},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm, often odd."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v > 64:
        v -= v % 64
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["quantize", "linear", "experts"])
    case = {"op": op, "dtype": rng.choice(["bf16", "fp16"])}
    if op == "quantize":
        cols = _spread(rng, 64, 28672)
        tokens = _spread(rng, 1, min(16384, (1 << 27) // cols))
        gather = rng.random() < 0.5
        rows = tokens * rng.choice([1, 2]) if gather else tokens
        case.update(tokens=tokens, rows=rows, cols=cols, gather=gather)
    elif op == "linear":
        m, n = _spread(rng, 1, 8192), _spread(rng, 64, 28672)
        case.update(m=m, n=n, k=_spread(rng, 64, 16384 if n <= 14336 else 8192), bias=rng.random() < 0.5)
    else:
        experts = rng.choice([4, 8, 16, 32, 60, 64, 128])
        n, k = _spread(rng, 256, 8192), _spread(rng, 256, 8192)
        most = 400_000_000 // experts
        if n * k > most:
            n = max(64, most // k)
        case.update(experts=experts, rows=_spread(rng, 1, 8192), pad=rng.choice([0, 0, 5, 130]), skew=rng.choice([0.0, 1.0, 3.0]),
                    n=n, k=k, bias=rng.random() < 0.5)
    return case


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _activation(g, rows, cols, dtype):
    """Normal values with a few channels far larger than the rest, as activations have them."""
    x = torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.float32)
    channels = torch.randint(0, cols, (max(1, cols // 1000),), generator=g, device="cuda")
    x[:, channels] *= 50.0
    return x.to(dtype)


def _codes(g, rows, cols, sigma, outliers=False):
    """Codes and scales of a quantized matrix, rows at a multiple of 16 bytes."""
    codes = torch.zeros(rows, (cols + 15) // 16 * 16, dtype=torch.int8, device="cuda")
    scales = torch.empty(rows, dtype=torch.float32, device="cuda")
    step = max(1, (1 << 26) // cols)
    for r in range(0, rows, step):
        x = torch.randn(min(step, rows - r), cols, generator=g, device="cuda", dtype=torch.float32) * sigma
        if outliers:
            x[:, :: 997] *= 50.0
        amax = x.abs().amax(1)
        codes[r:r + step, :cols] = torch.round(x * (127.0 / amax)[:, None]).to(torch.int8)
        scales[r:r + step] = amax / 127.0
    return codes[:, :cols], scales


def _counts(case, seed):
    """Rows of each expert: uneven, some empty where the routing is skewed."""
    g = torch.Generator()
    g.manual_seed(int(seed) * 7 + 1)
    p = torch.exp(case["skew"] * torch.randn(case["experts"], generator=g, dtype=torch.float64).clamp(-1.5, 1.0))
    picks = torch.multinomial(p, case["rows"], replacement=True, generator=g)
    return torch.bincount(picks, minlength=case["experts"])


def prepare(case, seed):
    g, dtype = _generator(seed), DTYPES[case["dtype"]]
    s = {"op": case["op"]}
    if case["op"] == "quantize":
        s["x"] = _activation(g, case["tokens"], case["cols"], dtype)
        s["index"] = None
        if case["gather"]:
            # every token goes to as many groups, in the groups' order
            s["index"] = (torch.randperm(case["rows"], generator=g, device="cuda") % case["tokens"]).to(torch.int32)
        wide = (case["cols"] + 15) // 16 * 16
        s["codes"] = torch.zeros(case["rows"], wide, dtype=torch.int8, device="cuda")[:, : case["cols"]]
        s["scales"] = torch.empty(case["rows"], dtype=torch.float32, device="cuda")
        if case["cols"] % 8:   # rows of the input at a multiple of 16 bytes too
            x = torch.zeros(case["tokens"], (case["cols"] + 7) // 8 * 8, dtype=dtype, device="cuda")
            x[:, : case["cols"]] = s["x"]
            s["x"] = x[:, : case["cols"]]
        return s
    n, k = case["n"], case["k"]
    groups = case.get("experts", 1)
    rows = case["m"] if case["op"] == "linear" else case["rows"] + case["pad"]
    s["a"], s["sa"] = _codes(g, rows, k, 1.0, outliers=True)
    w, sw = _codes(g, groups * n, k, 0.02)
    s["bias"] = torch.randn(groups, n, generator=g, device="cuda", dtype=torch.float32) * 0.1 if case["bias"] else None
    s["d"] = torch.zeros(rows, (n + 7) // 8 * 8, dtype=dtype, device="cuda")[:, :n]
    if case["op"] == "linear":
        s["w"], s["sw"] = w, sw
        s["bias"] = None if s["bias"] is None else s["bias"][0]
    else:
        s["w"], s["sw"] = w.unflatten(0, (groups, n)), sw.view(groups, n)
        counts = _counts(case, seed)
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(torch.int32).cuda()
        s["most"] = int(counts.max())   # what a padded product needs to know beforehand
    return s


def _plain_quantize(x, index):
    v = x.float() if index is None else x.float()[index.long()]
    amax = v.abs().amax(1)
    full = torch.where(amax > 0, amax, torch.full_like(amax, 127.0))
    return torch.round(v * 127.0 / full[:, None]).to(torch.int8), full / 127.0


def _plain_linear(a, sa, w, sw, bias, dtype):
    # whole-number sums pass 2^24: 64 bits hold them
    y = (a.double() @ w.double().T) * sa[:, None].double() * sw[None, :].double()
    if bias is not None:
        y = y + bias.double()
    return y.to(dtype)


def _plain_experts(a, sa, w, sw, offsets, bias, d, most):
    rows, experts = a.shape[0], w.shape[0]
    bounds = offsets.long()
    at = (bounds[:-1, None] + torch.arange(most, device=a.device)[None, :]).clamp(max=rows - 1)
    y = torch.bmm(a[at].double(), w.double().transpose(1, 2))            # every expert's rows, padded
    y = y * sa[at][:, :, None].double() * sw[:, None, :].double()
    if bias is not None:
        y = y + bias[:, None, :].double()
    r = torch.arange(rows, device=a.device)
    e = torch.searchsorted(bounds, r, right=True) - 1
    inside = (e >= 0) & (e < experts)
    e = e.clamp(0, experts - 1)
    picked = y[e, (r - bounds[e]).clamp(0, most - 1)].to(d.dtype)
    return torch.where(inside[:, None], picked, d)


def run(state):
    s = state
    if own:
        from block_scaled_fp4_05_b200 import fp4
        if s["op"] == "quantize":
            fp4.fp4_quantize_int8(s["x"], s["codes"], s["scales"], row_index=s["index"])
            return s["codes"], s["scales"]
        # the weights were quantized ahead of time
        kernel = fp4.GEMM_AUTO | fp4.GEMM_B_STATIC
        if s["op"] == "linear":
            fp4.fp4_gemm_int8(s["a"], s["sa"], s["w"], s["sw"], s["d"], bias=s["bias"], kernel=kernel)
        else:
            fp4.fp4_gemm_int8_grouped(s["a"], s["sa"], s["w"], s["sw"], s["offsets"], s["d"], bias=s["bias"], kernel=kernel)
        return s["d"]
    if s["op"] == "quantize":
        return _plain_quantize(s["x"], s["index"])
    if s["op"] == "linear":
        return _plain_linear(s["a"], s["sa"], s["w"], s["sw"], s["bias"], s["d"].dtype)
    return _plain_experts(s["a"], s["sa"], s["w"], s["sw"], s["offsets"], s["bias"], s["d"], s["most"])


def work(case):
    if case["op"] == "quantize":
        read = min(case["tokens"], case["rows"])
        return {"bytes": 2 * read * case["cols"] + case["rows"] * (case["cols"] + 4 + (4 if case["gather"] else 0)),
                "flops": 3 * case["rows"] * case["cols"]}
    n, k = case["n"], case["k"]
    rows = case["m"] if case["op"] == "linear" else case["rows"]
    # experts that rows reach, as many as even routing reaches in the mean
    active = 1 if case["op"] == "linear" else case["experts"] * (1 - (1 - 1 / case["experts"]) ** rows)
    channel = 4 + (4 if case["bias"] else 0)
    return {"bytes": rows * (k + 4 + 2 * n) + active * n * (k + channel) + (4 * (case["experts"] + 1) if case["op"] == "experts" else 0),
            "flops": 2 * rows * n * k}


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "quantize":
        x = s["x"] if s["index"] is None else torch.index_select(s["x"], 0, s["index"])
        codes, scales = torch.empty(x.shape, dtype=torch.int8, device="cuda"), []
        step = max(1, (1 << 26) // case["cols"])
        for r in range(0, x.shape[0], step):
            v = x[r:r + step].to(torch.float64)
            top = torch.maximum(v.max(1).values, -v.min(1).values)
            one = torch.where(top == 0, torch.ones_like(top), top / 127)
            # 127 x / amax: the quotient of the code's definition, halves to the even neighbour
            q = torch.where(top[:, None] == 0, torch.zeros_like(v), 127 * v / torch.where(top == 0, one, top)[:, None])
            codes[r:r + step] = q.round().to(torch.int8)
            scales.append(one)
        return codes, torch.cat(scales)
    if s["op"] == "linear":
        y = torch.empty(s["d"].shape, dtype=torch.float64, device="cuda")
        left = s["a"].to(torch.float64)
        for c in range(0, case["n"], 4096):
            right = s["w"][c:c + 4096].to(torch.float64) * s["sw"][c:c + 4096].to(torch.float64).unsqueeze(1)
            torch.mul(torch.mm(left, right.t()), s["sa"].to(torch.float64).unsqueeze(1), out=y[:, c:c + 4096])
        return y if s["bias"] is None else y.add_(s["bias"].to(torch.float64))
    y = s["d"].to(torch.float64)
    bounds = s["offsets"].tolist()
    for e in range(case["experts"]):
        lo, hi = bounds[e], bounds[e + 1]
        if lo < hi:
            left = s["a"][lo:hi].to(torch.float64) * s["sa"][lo:hi].to(torch.float64).unsqueeze(1)
            right = s["w"][e].to(torch.float64) * s["sw"][e].to(torch.float64).unsqueeze(1)
            y[lo:hi] = torch.mm(left, right.t())
            if s["bias"] is not None:
                y[lo:hi] += s["bias"][e].to(torch.float64)
    return y
