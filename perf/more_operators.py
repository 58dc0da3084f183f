"""The cases that the router, the NVFP4 matrix products and the AdamW step are measured on.

They close the loop around the quantizers in a training or serving step:

  router                 logits -> expert ids and weights (what the routing plan and the
                         combination take), and backwards the gradient of the logits
  gemm                   act(a b^T + bias) + residual of two NVFP4 operands; backwards the gradient
                         through the epilogue (the products of the backward pass are gemms again)
  gemm grouped           an expert's rows times that expert's weights, and the gradients of the
                         experts' weights from columnwise operands
  adamw                  the update of many tensors at once, its states in 32 or in 8 bits, with the
                         BF16 weights and their amax that the weight quantizer takes

`own` selects between the plain torch form and this package's kernels.
"""
import math

import torch

own = False

# ---- cases -------------------------------------------------------------------------------------


def _case(name, op, **kw):
    return dict(name=name, op=op, **kw)


def listed():
    return [
        # one decoding step of 16 sequences: sigmoid scores, a balance bias, 4 of 8 groups
        _case("router_decode_16_256experts", "router", tokens=16, experts=256, topk=8,
              score="sigmoid", groups=8, top_groups=4, bias=True, renorm=True, scale=2.5,
              dtype="float32"),
        # the routing of a large training batch over the benchmark's 64 experts
        _case("router_train_32768_64experts", "router", tokens=32768, experts=64, topk=8,
              score="softmax", groups=1, top_groups=1, bias=False, renorm=True, scale=1.0,
              dtype="bfloat16"),
        # the gradient of a training batch's logits
        _case("router_backward_16384_256experts", "router_backward", tokens=16384, experts=256,
              topk=8, score="sigmoid", groups=8, top_groups=4, bias=True, renorm=True, scale=2.5,
              dtype="float32"),
        # one token through the benchmark's weight matrix: latency and the bytes of the weights
        _case("gemm_1x14336x4096", "gemm", m=1, n=14336, k=4096, act="none", bias=False,
              residual=False, preact=False, amax=False, out="bfloat16"),
        # a ragged batch through an odd projection with the whole epilogue
        _case("gemm_1037x1000x2080", "gemm", m=1037, n=1000, k=2080, act="silu", bias=True,
              residual=True, preact=False, amax=True, out="bfloat16"),
        # the first projection of a training step's dense feed-forward layer at the benchmark's
        # activation and weight sizes, the pre-activation kept for the backward pass
        _case("gemm_8192x14336x4096", "gemm", m=8192, n=14336, k=4096, act="gelu", bias=True,
              residual=False, preact=True, amax=True, out="bfloat16"),
        # the gradient through that layer's epilogue
        _case("gemm_backward_8192x14336", "gemm_backward", m=8192, n=14336, act="gelu"),
        # a decoding step's rows through the gate and up projections of their experts: most experts
        # have a row or two, and their weights are what is read
        _case("grouped_decode_128rows_4096x7168", "grouped", rows=128, experts=128, active=80, n=4096,
              k=7168, live=1.0),
        # the packed tensor of the benchmark's grouped quantization through 64 experts
        _case("grouped_train_32768rows_4096x7168", "grouped", rows=32768, experts=64, active=60,
              n=4096, k=7168, live=0.98),
        # the gradient of 32 experts' down projections, kept in 32 bits
        _case("wgrad_32768rows_7168x2048", "wgrad", rows=32768, experts=32, active=32, n=7168, k=2048,
              live=1.0, out="float32"),
        # norms, biases and routers: many small tensors of odd sizes, states in 32 bits
        _case("adamw_97_small_tensors", "adamw", tensors=97, low=1, high=300000, bits=32,
              grad="float32"),
        # a layer's expert matrices with their states in 8 bits
        _case("adamw8_24_matrices", "adamw", tensors=24, low=4000000, high=16000000, bits=8,
              grad="bfloat16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


ACTS = ("none", "relu", "relu2", "gelu", "silu")


def draw(rng):
    op = rng.choice(["router", "router_backward", "gemm", "gemm", "gemm_backward", "grouped", "wgrad",
                     "adamw"])
    if op.startswith("router"):
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _log(rng, 4, 256 // groups)
        top_groups = rng.randint(max(1, groups // 2), groups)
        return dict(op=op, tokens=_log(rng, 1, 32768), experts=experts,
                    topk=rng.randint(1, min(8, experts // groups * top_groups)),
                    score=rng.choice(["softmax", "sigmoid"]), groups=groups, top_groups=top_groups,
                    bias=rng.choice([True, False]), renorm=rng.choice([True, False]),
                    scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["float32", "bfloat16"]))
    if op == "gemm":
        n, k = _log(rng, 8, 14336), 32 * _log(rng, 1, 448)
        m = _log(rng, 1, min(8192, 8192 * 14336 * 4096 // (n * k)))
        return dict(op=op, m=m, n=n, k=k, act=rng.choice(ACTS), bias=rng.choice([True, False]),
                    residual=rng.choice([True, False]), preact=rng.choice([True, False]),
                    amax=rng.choice([True, False]), out=rng.choice(["bfloat16", "bfloat16", "float32"]))
    if op == "gemm_backward":
        n = _log(rng, 8, 14336)
        return dict(op=op, m=_log(rng, 1, min(32768, 8192 * 14336 // n)), n=n, act=rng.choice(ACTS[1:]))
    if op in ("grouped", "wgrad"):
        experts = _log(rng, 1, 128)
        n, k = 8 * _log(rng, 4, 512), 32 * _log(rng, 4, 224 if op == "grouped" else 64)
        most = min(32768, 32768 * 4096 * 7168 // (4 * n * k))
        case = dict(op=op, rows=_log(rng, 1, most), experts=experts, active=rng.randint(1, experts), n=n,
                    k=k, live=rng.choice([1.0, 1.0, 0.9]))
        case["active"] = min(case["active"], max(1, int(case["rows"] * case["live"])))
        if op == "wgrad":
            case["out"] = rng.choice(["float32", "bfloat16"])
        return case
    high = _log(rng, 100, 8000000)
    return dict(op=op, tensors=_log(rng, 1, max(1, min(200, 100000000 // high))), low=max(1, high // 30),
                high=high, bits=rng.choice([32, 8]), grad=rng.choice(["float32", "bfloat16"]))


def _sizes(case):
    """Sizes of the tensors of an AdamW case: a fixed spread between `low` and `high`."""
    n, lo, hi = case["tensors"], math.log(case["low"]), math.log(case["high"])
    return [int(round(math.exp(lo + (hi - lo) * ((i * 0.6180339887) % 1.0)))) | 1 for i in range(n)]


def work(case):
    op = case["op"]
    if op.startswith("router"):
        T, E, K = case["tokens"], case["experts"], case["topk"]
        item = 4 if case["dtype"] == "float32" else 2
        if op == "router":
            return {"bytes": T * E * item + T * K * 8 + (4 * E if case["bias"] else 0),
                    "flops": 4 * T * E}
        dense = case["score"] == "softmax" and not case["renorm"]
        return {"bytes": T * (E if dense else K) * item + T * E * item + T * K * 8,
                "flops": 4 * T * (E if dense else K)}
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        out = 4 if case["out"] == "float32" else 2
        return {"bytes": (m + n) * k * 9 // 16 + m * n * (out + 2 * case["preact"] +
                                                           out * case["residual"]) + 2 * n * case["bias"],
                "flops": 2 * m * n * k}
    if op == "gemm_backward":
        return {"bytes": 6 * case["m"] * case["n"] + 4 * case["n"], "flops": 10 * case["m"] * case["n"]}
    if op in ("grouped", "wgrad"):
        live, n, k = int(case["rows"] * case["live"]), case["n"], case["k"]
        if op == "grouped":
            return {"bytes": (live + case["active"] * n) * k * 9 // 16 + 2 * case["rows"] * n,
                    "flops": 2 * live * n * k}
        return {"bytes": live * (n + k) * 9 // 16 +
                case["experts"] * n * k * (4 if case["out"] == "float32" else 2),
                "flops": 2 * live * n * k}
    total = sum(_sizes(case))
    each = 8 + 2 + (4 if case["grad"] == "float32" else 2)  # p read and written, the weight, the gradient
    each += 16 if case["bits"] == 32 else 4 + 4 / 32
    return {"bytes": int(total * each), "flops": 14 * total}


# ---- inputs ------------------------------------------------------------------------------------


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 29)
    return g


def _randn(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * std


def _quantized(x):
    """NVFP4 codes [R, C/2], scales [R, C/16] and [amax, S_dec] of x [R, C] float32."""
    R, C = x.shape
    amax = x.abs().amax().clamp_min(1e-30)
    enc = 2688.0 / amax
    b = x.reshape(R, C // 16, 16)
    scales = ((b.abs().amax(2) / 6) * enc).clamp_max(448).to(torch.float8_e4m3fn)
    s = scales.float()
    v = b * torch.where(s > 0, enc / s, 0).unsqueeze(2)
    step = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    code = torch.bucketize(v.abs(), step, out_int32=True).to(torch.uint8) + \
        (v < 0).to(torch.uint8) * 8
    code = code.reshape(R, C)
    return code[:, ::2] | (code[:, 1::2] << 4), scales.view(torch.uint8), torch.stack([amax, 1 / enc])


def _ends(case, g):
    """Expert ends of packed rows: `active` experts with a row at least, uneven, the others empty."""
    E, A, live = case["experts"], case["active"], int(case["rows"] * case["live"])
    live = max(live, 0)
    with_rows = torch.randperm(E, generator=g, device="cuda")[:A]
    p = torch.zeros(E, device="cuda", dtype=torch.float64)
    p[with_rows] = _randn(g, A, std=0.25).exp().double()
    counts = (p / p.sum() * max(live - A, 0)).floor().long()
    counts[with_rows] += min(1, live)
    counts = counts.tolist()
    first = int(with_rows[0])
    counts[first] += live - sum(counts)
    ends, at = [], 0
    for c in counts:
        at += c
        ends.append(at)
    return ends


def _dense(case, s, g):
    m, n, k = case["m"], case["n"], case["k"]
    s["a"] = _quantized(_randn(g, m, k))
    s["b"] = _quantized(_randn(g, n, k, std=k ** -0.5))
    s["bias"] = _randn(g, n, std=0.5).to(torch.bfloat16) if case["bias"] else None
    s["residual"] = _randn(g, m, n).to(getattr(torch, case["out"])) if case["residual"] else None


def _expert_operands(case, s, g):
    T, E, n, k = case["rows"], case["experts"], case["n"], case["k"]
    ends = _ends(case, g)
    s["offsets"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    begins = [0] + ends[:-1]
    s["most"] = max(e - b for b, e in zip(begins, ends))
    # the experts with rows (one at least), and each expert's place among them
    s["active"] = torch.tensor([e for e in range(E) if ends[e] > begins[e]] or [0], device="cuda")
    s["place"] = torch.zeros(E, dtype=torch.int64, device="cuda")
    s["place"][s["active"]] = torch.arange(s["active"].numel(), device="cuda")
    if case["op"] == "grouped":
        s["a"] = [torch.zeros(T, k // 2, dtype=torch.uint8, device="cuda"),
                  torch.zeros(T, k // 16, dtype=torch.uint8, device="cuda"),
                  torch.ones(E, 2, device="cuda")]
        s["b"] = [torch.empty(E, n, k // 2, dtype=torch.uint8, device="cuda"),
                  torch.empty(E, n, k // 16, dtype=torch.uint8, device="cuda"),
                  torch.empty(E, 2, device="cuda")]
        for e, (b, end) in enumerate(zip(begins, ends)):
            for to, v in zip(s["b"], _quantized(_randn(g, n, k, std=k ** -0.5))):
                to[e] = v
            if end > b:
                codes, scales, s["a"][2][e] = _quantized(_randn(g, end - b, k))
                s["a"][0][b:end], s["a"][1][b:end] = codes, scales
        return
    # columnwise operands of the grouped quantizer: an expert's tokens start at a multiple of 16
    cap = (T + 15 * E + 31) // 32 * 32
    s["starts"] = []
    for name, rows in (("a", n), ("b", k)):
        s[name] = [torch.zeros(rows, cap // 2, dtype=torch.uint8, device="cuda"),
                   torch.zeros(rows, cap // 16, dtype=torch.uint8, device="cuda"),
                   torch.ones(E, 2, device="cuda")]
        at = 0
        for e, (b, end) in enumerate(zip(begins, ends)):
            pad = (end - b + 15) // 16 * 16
            if name == "a":
                s["starts"].append(at)
            if pad:
                x = torch.zeros(rows, pad, device="cuda")
                x[:, :end - b] = _randn(g, rows, end - b, std=1.0 if name == "b" else 1e-3)
                codes, scales, s[name][2][e] = _quantized(x)
                s[name][0][:, at // 2:(at + pad) // 2] = codes
                s[name][1][:, at // 16:(at + pad) // 16] = scales
            at += pad


LR, BETAS, EPS, STEP = 3e-4, (0.9, 0.95), 1e-8, 40


def _flat(sizes, unit):
    """Places of tensors of these sizes one behind the other, each at a multiple of `unit`."""
    at, places = 0, []
    for n in sizes:
        places.append(at)
        at += (n + unit - 1) // unit * unit
    return places, at


def _optimizer(case, s, g, seed):
    """Tensors in flat buffers, each at a multiple of 64 elements, zeros between them."""
    sizes = _sizes(case)
    places, total = _flat(sizes, 64)
    s["sizes"], s["places"] = sizes, places
    block_tensor = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), torch.tensor(
        [(n + 63) // 64 * 2 for n in sizes], device="cuda"))
    s["block_tensor"] = block_tensor
    s["block_in_tensor"] = torch.arange(total // 32, device="cuda") - torch.tensor(
        places, device="cuda")[block_tensor] // 32
    inside = s["block_in_tensor"].unsqueeze(1) * 32 + torch.arange(32, device="cuda")
    inside = (inside < torch.tensor(sizes, device="cuda")[block_tensor].unsqueeze(1)).reshape(-1)
    # matrices decay, one tensor in five (norms and biases) does not
    s["decay"] = [0.0 if i % 5 == 0 else 0.1 for i in range(len(sizes))]
    s["block_decay"] = torch.tensor(s["decay"], device="cuda")[block_tensor]
    spread = _randn(g, total // 32, 1).exp().expand(-1, 32).reshape(-1) * 1e-3
    s["p"] = torch.where(inside, _randn(g, total, std=0.02), 0)
    s["grad"] = torch.where(inside, _randn(g, total) * spread, 0).to(getattr(torch, case["grad"]))
    m = torch.where(inside, _randn(g, total, std=0.3) * spread, 0)
    v = torch.where(inside, (_randn(g, total).square() * 0.5 + 0.3) * spread.square(), 0)
    s["weight"] = torch.zeros(total, dtype=torch.bfloat16, device="cuda")
    s["grad_scale"] = torch.full((1,), 0.75, device="cuda")  # from the clipping of the norm
    s["seed"] = seed + 1000
    if case["bits"] == 32:
        s["m"], s["v"] = m, v
    else:
        s["m"], s["m_scale"] = _keep8(m)
        s["v"], s["v_scale"] = _keep8(v.sqrt())
        s["m"], s["v"] = s["m"].view(torch.uint8), s["v"].view(torch.uint8)
    if own:
        from nvfp4_block_scaled_quantize_gb300 import api
        # the optimizer that a program makes once, over its parameters
        cut = lambda t: [t[at:at + n] for at, n in zip(places, sizes)]  # noqa: E731
        cut32 = lambda t: [t[at // 32:at // 32 + (n + 31) // 32] for at, n in zip(places, sizes)]  # noqa: E731
        state = dict(exp_avg=cut(s["m"]), exp_avg_sq=cut(s["v"]))
        if case["bits"] == 8:
            state.update(exp_avg_scales=cut32(s["m_scale"]), exp_avg_sq_scales=cut32(s["v_scale"]))
        s["optimizer"] = api.AdamW(cut(s["p"]), cut(s["grad"]), weights=cut(s["weight"]),
                                   weight_decay=s["decay"], betas=BETAS, eps=EPS,
                                   state_bits=case["bits"], state=state)


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = {"case": case}
    if op.startswith("router"):
        T, E = case["tokens"], case["experts"]
        s["logits"] = (_randn(g, T, E) + _randn(g, E, std=0.5)).to(getattr(torch, case["dtype"]))
        s["bias"] = _randn(g, E, std=0.05) if case["bias"] else None
        if op == "router_backward":
            s["ids"] = _choose(s)[0].to(torch.int32)
            s["grad"] = _randn(g, T, case["topk"], std=1e-2)
    elif op == "gemm":
        _dense(case, s, g)
    elif op == "gemm_backward":
        s["grad"] = _randn(g, case["m"], case["n"], std=1e-3).to(torch.bfloat16)
        s["preact"] = _randn(g, case["m"], case["n"], std=1.5).to(torch.bfloat16)
    elif op in ("grouped", "wgrad"):
        _expert_operands(case, s, g)
    else:
        _optimizer(case, s, g, seed)
    return s


# ---- plain forms -------------------------------------------------------------------------------


def _scores(s):
    """Scores in 64 bits: the order of the choices depends on differences of their last bits."""
    x = s["logits"].double()
    return torch.softmax(x, 1) if s["case"]["score"] == "softmax" else torch.sigmoid(x)


def _choose(s):
    """(ids, scores) of the chosen experts, best first, ties to the lowest index."""
    case = s["case"]
    T, E, G = case["tokens"], case["experts"], case["groups"]
    score = _scores(s)
    # without a bias the order of the scores is that of the logits
    choice = s["logits"].double() if s["bias"] is None else score + s["bias"].double()
    if case["top_groups"] < G:
        by_group = (score if s["bias"] is None else choice).reshape(T, G, E // G)
        rank = by_group.topk(min(2, E // G), dim=2).values.sum(2)
        best = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        held = torch.zeros(T, G, dtype=torch.bool, device="cuda").scatter_(1, best, True)
        choice = torch.where(held.repeat_interleave(E // G, dim=1), choice, -math.inf)
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :case["topk"]]
    return ids, score.gather(1, ids)


def _router(s):
    ids, w = _choose(s)
    if s["case"]["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": (w * s["case"]["scale"]).float()}


def _router_backward(s):
    case = s["case"]
    p, ids, g = _scores(s), s["ids"].long(), s["grad"].double() * case["scale"]
    w = p.gather(1, ids)
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        g = (g - (g * w).sum(1, keepdim=True) / total) / total
    d = torch.zeros_like(p).scatter_(1, ids, g)
    if case["score"] == "sigmoid":
        d = d * p * (1 - p)
    elif case["renorm"]:  # the part that all logits share cancels
        d = d * p
    else:
        d = p * (d - (d * p).sum(1, keepdim=True))
    return {"grad_logits": d.to(s["logits"].dtype)}


def _pairs():
    one = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda")
    one = torch.cat([one, -one])
    return torch.stack([one.repeat(16), one.repeat_interleave(16)], 1)


def _values(codes, scales):
    """What codes [.., C/2] and scales [.., C/16] stand for, but for the global scale."""
    v = _pairs()[codes.int()].reshape(*codes.shape[:-1], -1, 16)
    return (v * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)).reshape(
        *codes.shape[:-1], -1)


def _act(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "relu2":
        return z.clamp_min(0).square()
    if act == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z * torch.sigmoid(z) if act == "silu" else z


def _slope(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "relu2":
        return 2 * z.clamp_min(0)
    if act == "gelu":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    p = torch.sigmoid(z)
    return p * (1 + z * (1 - p))


def _gemm(s):
    case = s["case"]
    z = (_values(*s["a"][:2]) @ _values(*s["b"][:2]).t()) * (s["a"][2][1] * s["b"][2][1])
    if s["bias"] is not None:
        z = z + s["bias"].float()
    out = _act(z, case["act"])
    if s["residual"] is not None:
        out = out + s["residual"].float()
    got = {"out": out.to(getattr(torch, case["out"]))}
    if case["preact"]:
        got["preact"] = z.to(torch.bfloat16)
    if case["amax"]:  # a BF16 output's maximum is a BF16 value
        got["amax"] = got["out"].abs().amax().reshape(1)
    return got


def _gemm_backward(s):
    g = s["grad"].float() * _slope(s["preact"].float(), s["case"]["act"])
    d = g.to(torch.bfloat16)
    return {"grad_preact": d, "grad_bias": g.sum(0), "amax": d.abs().amax().reshape(1)}


def _places(s):
    """Each packed row's expert (the last one's for rows behind the end), place in it, and whether it
    is live."""
    rows, offsets = s["case"]["rows"], s["offsets"].long()
    at = torch.arange(rows, device="cuda")
    expert = torch.searchsorted(offsets, at, right=True).clamp_max(offsets.numel() - 1)
    begins = torch.cat([torch.zeros_like(offsets[:1]), offsets[:-1]])
    return expert, at - begins[expert], at < offsets[-1]


def _grouped(s):
    case = s["case"]
    expert, place, live = _places(s)
    place = torch.where(live, place, s["most"])  # a row of padding behind the longest
    active, expert = s["active"], s["place"][expert]
    x = torch.zeros(active.numel(), s["most"] + 1, case["k"], device="cuda")
    x[expert, place] = torch.where(live.unsqueeze(1), _values(*s["a"][:2]), 0)
    y = torch.bmm(x, _values(s["b"][0][active], s["b"][1][active]).transpose(1, 2))
    y = y * (s["a"][2][active, 1] * s["b"][2][active, 1]).reshape(-1, 1, 1)
    return {"out": torch.where(live.unsqueeze(1), y[expert, place], 0).to(torch.bfloat16)}


def _wgrad(s):
    case, offsets, active = s["case"], s["offsets"].long(), s["active"]
    counts = torch.diff(offsets, prepend=torch.zeros_like(offsets[:1]))
    pads = (counts + 15) // 16 * 16
    starts, pads = (pads.cumsum(0) - pads)[active], pads[active]
    at = torch.arange((s["most"] + 15) // 16 * 16, device="cuda")
    inside = at < pads.unsqueeze(1)
    at = torch.where(inside, starts.unsqueeze(1) + at, 0)
    a, b = ((_values(*s[x][:2])[:, at] * inside).transpose(0, 1) for x in ("a", "b"))
    d = torch.bmm(a, b.transpose(1, 2))
    d = d * (s["a"][2][active, 1] * s["b"][2][active, 1]).reshape(-1, 1, 1)
    out = torch.zeros(case["experts"], case["n"], case["k"], dtype=getattr(torch, case["out"]),
                      device="cuda")
    out[active] = d.to(out.dtype)
    return {"out": out}


def _scale_of(top):
    """The exponent e of the smallest 2^e, e >= -127, with top <= 448 * 2^e."""
    m, e = torch.frexp(top)
    e = torch.where(m > 0.875, e - 8, e - 9)
    return torch.where(m == 0, -127, e).clamp_min(-127)


def _keep8(x):
    """E4M3 codes and E8M0 scales of blocks of 32, rounded to nearest."""
    b = x.reshape(-1, 32)
    e = _scale_of(b.abs().amax(1))
    codes = torch.ldexp(b, -e.unsqueeze(1)).to(torch.float8_e4m3fn)
    return codes.reshape(-1), (e + 127).to(torch.uint8)


def _back8(codes, scales):
    v = codes.view(torch.float8_e4m3fn).float().reshape(-1, 32)
    return torch.ldexp(v, scales.to(torch.int32).unsqueeze(1) - 127).reshape(-1)


def _philox(counter, key):
    """Philox4x32-10 of int64 tensors holding 32-bit words."""
    low = 0xFFFFFFFF
    c, (k0, k1) = counter, key
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((b >> 32) & low) ^ c[1] ^ k0, b & low, ((a >> 32) & low) ^ c[3] ^ k1, a & low]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return c


def _random16(s):
    """The 16 random bits of each element: eight elements share a draw, each takes half a word, the
    low half first; the counter is (index of the eight, its high word, the tensor, the step)."""
    j = (s["block_in_tensor"].unsqueeze(1) * 4 + torch.arange(4, device="cuda")).reshape(-1)
    tensor = s["block_tensor"].repeat_interleave(4)
    words = _philox([j & 0xFFFFFFFF, j >> 32, tensor, torch.full_like(tensor, STEP)],
                    (s["seed"] & 0xFFFFFFFF, s["seed"] >> 32))
    words = torch.stack(words, 1)
    return torch.stack([words & 0xFFFF, words >> 16], 2).reshape(-1)


def _keep8_random(x, random):
    """The same of values >= 0, rounded up with the probability of the part above the code below;
    what is not zero keeps the smallest code at least."""
    b = x.reshape(-1, 32)
    e = _scale_of(b.amax(1))
    t = torch.ldexp(b, -e.unsqueeze(1))
    step = (torch.frexp(t)[1] - 1).clamp_min(-6) - 3
    q = torch.floor(torch.ldexp(t, -step) + random.reshape(-1, 32) / 65536.0)
    q = torch.where(t > 0, q.clamp_min(1), q)
    codes = torch.ldexp(q, step).to(torch.float8_e4m3fn)
    return codes.reshape(-1), (e + 127).to(torch.uint8)


def _adamw(s):
    case = s["case"]
    b1, b2 = BETAS
    eight = case["bits"] == 8
    g = s["grad"].float() * s["grad_scale"]
    m = _back8(s["m"], s["m_scale"]) if eight else s["m"]
    v = _back8(s["v"], s["v_scale"]).square() if eight else s["v"]
    m = m * b1 + g * (1 - b1)
    v = v * b2 + (g * g) * (1 - b2)
    root = v.sqrt()
    update = (m * (LR / (1 - b1 ** STEP))) / (root * (1 - b2 ** STEP) ** -0.5 + EPS)
    keep = (1 - LR * s["block_decay"]).unsqueeze(1)
    s["p"].copy_((s["p"].reshape(-1, 32) * keep).reshape(-1) - update)
    s["weight"].copy_(s["p"])
    if eight:
        codes, scales = _keep8(m)
        s["m"].copy_(codes.view(torch.uint8))
        s["m_scale"].copy_(scales)
        codes, scales = _keep8_random(root, _random16(s))
        s["v"].copy_(codes.view(torch.uint8))
        s["v_scale"].copy_(scales)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    top = torch.zeros(len(s["sizes"]), device="cuda")
    top.scatter_reduce_(0, s["block_tensor"], s["weight"].reshape(-1, 32).abs().amax(1).float(), "amax")
    return _updated(s, top)


def _updated(s, amax):
    got = {"p": s["p"], "weight": s["weight"], "amax": amax.to(torch.bfloat16)}
    if s["case"]["bits"] == 32:
        return dict(got, m=s["m"], v=s["v"])
    return dict(got, m=s["m"].view(torch.float8_e4m3fn), v=s["v"].view(torch.float8_e4m3fn),
                m_scale=s["m_scale"], v_scale=s["v_scale"])


# ---- the package's operators -------------------------------------------------------------------


def _run_own(s):
    from nvfp4_block_scaled_quantize_gb300 import api
    case, op = s["case"], s["case"]["op"]
    if op == "router":
        ids, weights = api.nvfp4_moe_router(s["logits"], case["topk"], score=case["score"],
                                            bias=s["bias"], groups=case["groups"],
                                            top_groups=case["top_groups"],
                                            renormalize=case["renorm"], scale=case["scale"])
        return {"ids": ids, "weights": weights}
    if op == "router_backward":
        return {"grad_logits": api.nvfp4_moe_router_backward(
            s["grad"], s["logits"], s["ids"], score=case["score"], renormalize=case["renorm"],
            scale=case["scale"])}
    if op == "gemm":
        got = api.nvfp4_gemm(*s["a"], *s["b"], bias=s["bias"], activation=case["act"],
                             residual=s["residual"], out_dtype=getattr(torch, case["out"]),
                             keep_preact=case["preact"], with_amax=case["amax"])
        if case["amax"]:
            got["amax"] = got["amax"].to(got["out"].dtype)
        return got
    if op == "gemm_backward":
        d, grad_bias, amax = api.nvfp4_gemm_epilogue_backward(s["grad"], s["preact"], case["act"])
        return {"grad_preact": d, "grad_bias": grad_bias, "amax": amax.to(torch.bfloat16)}
    if op == "grouped":
        return {"out": api.nvfp4_gemm_grouped(*s["a"], *s["b"], s["offsets"])["out"]}
    if op == "wgrad":
        return {"out": api.nvfp4_gemm_grouped_wgrad(*s["a"], *s["b"], s["offsets"],
                                                    out_dtype=getattr(torch, case["out"]))}
    amax = s["optimizer"].step(lr=LR, step=STEP, grad_scale=s["grad_scale"], seed=s["seed"])
    return _updated(s, amax)


PLAIN = {"router": _router, "router_backward": _router_backward, "gemm": _gemm,
         "gemm_backward": _gemm_backward, "grouped": _grouped, "wgrad": _wgrad, "adamw": _adamw}


def run(state):
    return _run_own(state) if own else PLAIN[state["case"]["op"]](state)


# ---- 64 bits -----------------------------------------------------------------------------------


def _operand64(codes, scales):
    """E2M1 by its fields (sign, two exponent bits, one of mantissa), times the block's scale."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(torch.int16)
    e, f = (c >> 1) & 3, (c & 1).double()
    v = torch.where(e == 0, f / 2, (1 + f / 2) * torch.exp2(e.double() - 1))
    v = torch.where(c >= 8, -v, v)
    return v * scales.view(torch.float8_e4m3fn).double().repeat_interleave(16, dim=-1)


def _act64(z, act):
    if act.startswith("relu"):
        return torch.where(z > 0, z, 0) ** (2 if act == "relu2" else 1)
    if act == "gelu":  # (1 + tanh(u)) / 2 = 1 / (1 + exp(-2u))
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z / (1 + torch.exp(-z)) if act == "silu" else z


def _exact_router(s):
    case = s["case"]
    x = s["logits"].double()
    if case["score"] == "softmax":
        t = torch.exp(x - x.amax(1, keepdim=True))
        p = t / t.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-x))
    K = case["topk"]
    if case["op"] == "router":
        T, E, G = case["tokens"], case["experts"], case["groups"]
        choice = p + (0 if s["bias"] is None else s["bias"].double())
        left = choice.clone()
        if case["top_groups"] < G:
            size = E // G
            best = left.reshape(T, G, size).sort(2, descending=True).values[:, :, :2].sum(2)
            order = best.argsort(1, descending=True)
            for j in range(case["top_groups"], G):
                out = order[:, j:j + 1] * size + torch.arange(size, device="cuda")
                left.scatter_(1, out, -math.inf)
        w = []
        for _ in range(K):
            at = left.argmax(1, keepdim=True)
            w.append(p.gather(1, at))
            left.scatter_(1, at, -math.inf)
        w = torch.cat(w, 1)
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return {"ids": None, "weights": w * case["scale"]}
    ids, g = s["ids"].long(), s["grad"].double() * case["scale"]
    picked = torch.zeros_like(p, dtype=torch.bool).scatter_(1, ids, True)
    dw = torch.zeros_like(p).scatter_(1, ids, g)
    q = torch.where(picked, p, 0)
    if case["renorm"]:  # w = q / sum q
        w = q / q.sum(1, keepdim=True)
        dw = (dw - (dw * w).sum(1, keepdim=True)) / q.sum(1, keepdim=True)
    dw = torch.where(picked, dw, 0)
    if case["score"] == "sigmoid":
        return {"grad_logits": dw * p * (1 - p)}
    shared = 0 if case["renorm"] else (dw * p).sum(1, keepdim=True)
    return {"grad_logits": p * dw - p * shared}


def _exact_adamw(s):
    b1, b2 = BETAS
    eight = s["case"]["bits"] == 8
    g = s["grad"].double() * 0.75

    def held(codes, scales):
        return codes.view(torch.float8_e4m3fn).double() * torch.exp2(
            scales.double() - 127).repeat_interleave(32)

    m = held(s["m"], s["m_scale"]) if eight else s["m"].double()
    v = held(s["v"], s["v_scale"]) ** 2 if eight else s["v"].double()
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g ** 2
    hat_m, hat_v = m / (1 - b1 ** STEP), v / (1 - b2 ** STEP)
    decay = s["block_decay"].double().repeat_interleave(32)
    p = s["p"].double()
    p = p - LR * decay * p - LR * hat_m / (hat_v.sqrt() + EPS)
    top = [p[at:at + n].abs().amax() for at, n in zip(s["places"], s["sizes"])]
    got = {"p": p, "weight": p, "amax": torch.stack(top)}
    if eight:
        b = m.reshape(-1, 32)
        f, e = torch.frexp(b.abs().amax(1, keepdim=True) / 448)
        e = torch.where(f == 0.5, e - 1, e).clamp_min(-127).double()
        t = b / torch.exp2(e)
        step = torch.exp2(torch.frexp(t)[1].double().sub(1).clamp_min(-6) - 3)
        return dict(got, m=(torch.round(t / step) * step).reshape(-1), v=None, m_scale=None, v_scale=None)
    return dict(got, m=m, v=v)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("router"):
        return _exact_router(s)
    if op == "gemm":
        z = _operand64(*s["a"][:2]) @ _operand64(*s["b"][:2]).t()
        z = z * s["a"][2][1].double() * s["b"][2][1].double()
        if s["bias"] is not None:
            z += s["bias"].double()
        out = _act64(z, case["act"])
        if s["residual"] is not None:
            out = out + s["residual"].double()
        got = {"out": out}
        if case["preact"]:
            got["preact"] = z
        if case["amax"]:
            got["amax"] = out.abs().amax().reshape(1)
        return got
    if op == "gemm_backward":
        z = s["preact"].double().requires_grad_()
        _act64(z, case["act"]).backward(s["grad"].double())
        return {"grad_preact": z.grad, "grad_bias": z.grad.sum(0), "amax": z.grad.abs().amax().reshape(1)}
    if op == "adamw":
        return _exact_adamw(s)
    ends = s["offsets"].tolist()
    scale = s["a"][2][:, 1].double() * s["b"][2][:, 1].double()
    if op == "grouped":
        out = torch.zeros(case["rows"], case["n"], dtype=torch.float64, device="cuda")
        begin = 0
        for e, end in enumerate(ends):
            if end > begin:
                w = _operand64(s["b"][0][e], s["b"][1][e])
                out[begin:end] = _operand64(s["a"][0][begin:end], s["a"][1][begin:end]) @ w.t() * scale[e]
            begin = end
        return {"out": out}
    out = torch.zeros(case["experts"], case["n"], case["k"], dtype=torch.float64, device="cuda")
    begin = 0
    for e, end in enumerate(ends):
        at, pad = s["starts"][e], (end - begin + 15) // 16 * 16
        if pad:
            a, b = (_operand64(s[x][0][:, at // 2:(at + pad) // 2].contiguous(),
                               s[x][1][:, at // 16:(at + pad) // 16].contiguous()) for x in ("a", "b"))
            out[e] = a @ b.t() * scale[e]
        begin = end
    return {"out": out}
