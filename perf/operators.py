"""The cases that the MoE routing and 8-bit checkpoint operators are measured on.

The operators sit on both sides of the grouped NVFP4 quantizer in a training or serving step of a
mixture-of-experts layer:

  plan                 expert ids [T, K] -> the packed order of the (token, choice) slots
  dispatch             token rows copied into that order (with the per-expert amax), and back-
                       wards the sum of a token's packed gradients
  combine              the weighted sum of a token's expert outputs, and backwards the packed
                       gradients and the gradients of the weights
  swiglu checkpoint    silu(gate) * up, its inputs kept in 8 bits, and the backward pass from them
  rmsnorm checkpoint   the norm, its input kept in 8 bits, and the backward pass from it

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
        # one decoding step of a batch of 16 sequences, 256 experts: all latency
        _case("plan_decode_16x8_256experts", "plan", tokens=16, topk=8, experts=256, drop=0.0,
              ids="int64"),
        # the routing of a large training batch over the benchmark's 64 experts, some slots dropped
        _case("plan_train_32768x8_64experts", "plan", tokens=32768, topk=8, experts=64, drop=0.02,
              ids="int32"),
        # one token of one sequence sent to its experts: the smallest serving call
        _case("dispatch_1x8_h7168", "dispatch", tokens=1, topk=8, experts=256, hidden=7168,
              drop=0.0),
        # the packed [32768, 7168] tensor that the benchmark's grouped quantization reads
        _case("dispatch_4096x8_h7168", "dispatch", tokens=4096, topk=8, experts=64, hidden=7168,
              drop=0.0),
        # a ragged batch under a capacity limit: odd sizes, some tokens lose slots
        _case("dispatch_backward_3001x6_h2056", "dispatch_backward", tokens=3001, topk=6,
              experts=37, hidden=2056, drop=0.06),
        # a small decoding batch's expert outputs summed
        _case("combine_24x8_h7168", "combine", tokens=24, topk=8, experts=256, hidden=7168,
              drop=0.0),
        # a training step's expert outputs summed, four experts a token
        _case("combine_8192x4_h4096", "combine", tokens=8192, topk=4, experts=64, hidden=4096,
              drop=0.0),
        # the gradient of the combination at the benchmark's size, some slots dropped
        _case("combine_backward_4096x8_h7168", "combine_backward", tokens=4096, topk=8,
              experts=64, hidden=7168, drop=0.02),
        # a ragged batch through a narrow expert, few live rows
        _case("swiglu_checkpoint_1037x1056", "swiglu_checkpoint", rows=1037, width=1056,
              experts=7, live=0.9),
        # the backward pass of a training step's packed expert rows
        _case("swiglu_checkpoint_backward_32768x2048", "swiglu_checkpoint_backward", rows=32768,
              width=2048, experts=64, live=0.98),
        # the activation tensor of the benchmark through its norm
        _case("rmsnorm_checkpoint_8192x4096", "rmsnorm_checkpoint", rows=8192, width=4096),
        # the gradient tensor of the benchmark back through its norm, with the residual's gradient
        _case("rmsnorm_checkpoint_backward_16384x8192", "rmsnorm_checkpoint_backward", rows=16384,
              width=8192, residual=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "dispatch", "dispatch_backward", "combine", "combine_backward",
                     "swiglu_checkpoint", "swiglu_checkpoint_backward", "rmsnorm_checkpoint",
                     "rmsnorm_checkpoint_backward"])
    if op == "plan":
        topk = rng.randint(1, 8)
        return dict(op=op, tokens=_log(rng, 1, 32768), topk=topk,
                    experts=_log(rng, max(topk, 2), 256), drop=rng.choice([0.0, 0.0, 0.03, 0.3]),
                    ids=rng.choice(["int32", "int64"]))
    if op.startswith(("dispatch", "combine")):
        topk = rng.randint(1, 8)
        hidden = 8 * _log(rng, 8, 1024)
        tokens = _log(rng, 1, min(16384, (4096 * 8 * 7168) // (topk * hidden)))
        return dict(op=op, tokens=tokens, topk=topk, experts=_log(rng, max(topk, 2), 256),
                    hidden=hidden, drop=rng.choice([0.0, 0.0, 0.03, 0.3]))
    width = 32 * _log(rng, 1, 512 if op.startswith("rmsnorm") else 128)
    if op.startswith("swiglu"):
        rows = _log(rng, 1, min(32768, 32768 * 2048 // width))
        return dict(op=op, rows=rows, width=width, experts=_log(rng, 1, 256),
                    live=rng.choice([1.0, 1.0, 0.97, 0.6]))
    rows = _log(rng, 1, min(32768, 16384 * 8192 // width))
    case = dict(op=op, rows=rows, width=width)
    if op == "rmsnorm_checkpoint_backward":
        case["residual"] = rng.choice([True, False])
    return case


def work(case):
    op = case["op"]
    if "tokens" in case:
        T, K, E, H = case["tokens"], case["topk"], case["experts"], case.get("hidden", 0)
        kept = T * K * (1 - case["drop"])
        if op == "plan":
            return {"bytes": T * K * ((8 if case["ids"] == "int64" else 4) + 8) + 4 * E, "flops": 0}
        if op == "dispatch":
            return {"bytes": 2 * T * H + 2 * T * K * H + 4 * T * K + 8 * E, "flops": 0}
        if op == "dispatch_backward":
            return {"bytes": 2 * kept * H + 2 * T * H + 4 * T * K, "flops": kept * H}
        if op == "combine":
            return {"bytes": 2 * kept * H + 2 * T * H + 8 * T * K, "flops": 2 * kept * H}
        return {"bytes": 2 * T * H + 2 * kept * H + 2 * T * K * H + 12 * T * K,
                "flops": 3 * kept * H}
    M, N = case["rows"], case["width"]
    if op.startswith("swiglu"):
        live = int(M * case["live"])
        ckpt = 2 * N + 2 * N // 32
        if op == "swiglu_checkpoint":  # h read; y, codes and scales written
            return {"bytes": 4 * N * live + (2 * N + ckpt) * M + 8 * case["experts"],
                    "flops": 8 * N * live}
        return {"bytes": (2 * N + ckpt) * live + 4 * N * M + 4 * case["experts"],
                "flops": 16 * N * live}
    ckpt = N + N // 32
    if op == "rmsnorm_checkpoint":
        return {"bytes": M * (2 * N + 2 * N + ckpt + 4) + 2 * N + 4, "flops": 5 * M * N}
    extra = 2 * N if case["residual"] else 0
    return {"bytes": M * (2 * N + ckpt + 2 * N + extra + 4) + 6 * N, "flops": 9 * M * N}


# ---- inputs ------------------------------------------------------------------------------------


def _normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _with_outliers(g, *shape):
    """Activations: N(0, 1), one in a thousand 100 times larger."""
    x = torch.randn(*shape, generator=g, device="cuda")
    far = torch.rand(*shape, generator=g, device="cuda") < 1e-3
    return torch.where(far, x * 100, x).to(torch.bfloat16)


def _expert_ids(case, g):
    """Top-k choices of a router with uneven experts (popularity log-normal); dropped slots are -1."""
    T, K, E = case["tokens"], case["topk"], case["experts"]
    logits = torch.randn(T, E, generator=g, device="cuda") + torch.randn(E, generator=g,
                                                                         device="cuda")
    top, ids = logits.topk(K, dim=1)
    weights = torch.softmax(top, dim=1)
    if case["drop"]:
        ids = torch.where(torch.rand(T, K, generator=g, device="cuda") < case["drop"], -1, ids)
    return ids, weights


def _offsets(case, g):
    """Expert ends of packed rows, the last `1 - live` of the rows belonging to no expert."""
    live = int(case["rows"] * case["live"])
    p = torch.randn(case["experts"], generator=g, device="cuda").exp()
    ends = (p.cumsum(0) / p.sum() * live).round().to(torch.int32)
    ends[-1] = live
    return ends


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    op = case["op"]
    s = {"case": case}
    if "tokens" in case:
        T, K, H = case["tokens"], case["topk"], case.get("hidden", 0)
        ids, weights = _expert_ids(case, g)
        if op == "plan":
            s["ids"] = ids.to(getattr(torch, case["ids"]))
            return s
        s["plan"] = _plan(ids, case["experts"])
        if op == "dispatch":
            s["x"] = _with_outliers(g, T, H)
        elif op == "dispatch_backward":
            s["grad"] = _normal(g, T * K, H, std=1e-3)
        else:
            s["weights"] = weights
            s["y"] = _normal(g, T * K, H)
            if op == "combine_backward":
                s["grad"] = _normal(g, T, H, std=1e-3)
        return s
    M, N = case["rows"], case["width"]
    if op.startswith("swiglu"):
        h = _with_outliers(g, M, 2 * N)
        s["offsets"] = _offsets(case, g)
    else:
        h = _with_outliers(g, M, N)
        s["weight"] = (1 + 0.3 * torch.randn(N, generator=g, device="cuda")).to(torch.bfloat16)
    if not op.endswith("backward"):
        s["x"] = h
        return s
    s["codes"], s["scales"] = _keep8(h)
    if op.startswith("rmsnorm"):
        s["rstd"] = torch.rsqrt(h.float().square().mean(1) + EPS)
        if case["residual"]:
            s["residual"] = _normal(g, M, N, std=1e-3)
    s["grad"] = _normal(g, M, N, std=1e-3)
    return s


# ---- plain forms -------------------------------------------------------------------------------

EPS = 1e-6


def _plan(ids, experts):
    flat = ids.reshape(-1).to(torch.int64)
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    order = torch.argsort(key, stable=True)
    counts = torch.zeros(experts + 1, dtype=torch.int64, device=ids.device)
    counts.scatter_add_(0, key, torch.ones_like(key))
    offsets = counts[:experts].cumsum(0)
    at = torch.arange(n, device=ids.device)
    rows = torch.empty_like(order)
    rows[order] = at
    rows = torch.where(key < experts, rows, -1)
    slots = torch.where(at < offsets[-1], order, -1)
    return {"row_of_slot": rows.to(torch.int32).reshape(ids.shape),
            "slot_of_row": slots.to(torch.int32), "offsets": offsets.to(torch.int32)}


def _expert_amax(rows, offsets):
    """max |.| of each expert's rows (0 for an expert without rows)."""
    n, E = rows.shape[0], offsets.numel()
    of = torch.searchsorted(offsets, torch.arange(n, device=rows.device, dtype=torch.int32),
                            right=True)
    top = torch.zeros(E + 1, dtype=torch.float32, device=rows.device)
    top.scatter_reduce_(0, of, rows.abs().amax(1).float(), "amax")
    return top[:E]


def _keep8(x):
    """E4M3 codes and E8M0 scales of blocks of 32: the smallest power of two that keeps the
    block's largest magnitude within 448."""
    M, N = x.shape
    b = x.float().reshape(M, N // 32, 32)
    m, e = torch.frexp(b.abs().amax(2))
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(m == 0, -127, e).clamp_min(-127)
    codes = torch.ldexp(b, -e.unsqueeze(2)).to(torch.float8_e4m3fn)
    return codes.reshape(M, N).view(torch.uint8), (e + 127).to(torch.uint8)


def _back(codes, scales):
    M, N = codes.shape
    v = codes.view(torch.float8_e4m3fn).float().reshape(M, N // 32, 32)
    return torch.ldexp(v, scales.to(torch.int32).unsqueeze(2) - 127).reshape(M, N)


def _live(s, rows):
    return (torch.arange(rows, device="cuda") < s["offsets"][-1]).unsqueeze(1)


def _run_plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "plan":
        return _plan(s["ids"], case["experts"])
    if "tokens" in case:
        plan = s["plan"]
        rows = plan["row_of_slot"].long()
        held = rows >= 0
        if op == "dispatch":
            slots = plan["slot_of_row"].long()
            token = slots.clamp_min(0) // case["topk"]
            packed = torch.where((slots >= 0).unsqueeze(1), s["x"][token], 0)
            return {"packed": packed, "amax": _expert_amax(packed, plan["offsets"])}
        if op == "dispatch_backward":
            v = torch.where(held.unsqueeze(2), s["grad"][rows.clamp_min(0)].float(), 0)
            return {"grad_x": v.sum(1).to(torch.bfloat16)}
        v = torch.where(held.unsqueeze(2), s["y"][rows.clamp_min(0)].float(), 0)
        w = torch.where(held, s["weights"], 0).unsqueeze(2)
        if op == "combine":
            return {"out": (v * w).sum(1).to(torch.bfloat16)}
        grad = s["grad"].float().unsqueeze(1)
        grad_w = (v * grad).sum(2)
        slots = plan["slot_of_row"].long()
        at = slots.clamp_min(0)
        grad_y = s["weights"].reshape(-1)[at].unsqueeze(1) * s["grad"][at // case["topk"]].float()
        grad_y = torch.where((slots >= 0).unsqueeze(1), grad_y, 0).to(torch.bfloat16)
        return {"grad_y": grad_y, "grad_weights": grad_w}
    M, N = case["rows"], case["width"]
    if op == "swiglu_checkpoint":
        h = torch.where(_live(s, M), s["x"], 0)
        codes, scales = _keep8(h)
        a, b = h[:, :N].float(), h[:, N:].float()
        y = (a * torch.sigmoid(a) * b).to(torch.bfloat16)
        return {"y": y, "codes": codes.view(torch.float8_e4m3fn), "scales": scales,
                "amax": _expert_amax(y, s["offsets"])}
    if op == "swiglu_checkpoint_backward":
        h = _back(s["codes"], s["scales"])
        a, b = h[:, :N], h[:, N:]
        g = s["grad"].float()
        p = torch.sigmoid(a)
        d = torch.cat([g * b * (p * (1 + a * (1 - p))), g * (a * p)], 1)
        return {"grad_h": torch.where(_live(s, M), d, 0).to(torch.bfloat16)}
    if op == "rmsnorm_checkpoint":
        x = s["x"].float()
        codes, scales = _keep8(s["x"])
        rstd = torch.rsqrt(x.square().mean(1) + EPS)
        y = (s["weight"].float() * (x * rstd.unsqueeze(1))).to(torch.bfloat16)
        return {"y": y, "codes": codes.view(torch.float8_e4m3fn), "scales": scales, "rstd": rstd,
                "amax": y.abs().amax().float().reshape(1)}
    r = s["rstd"].unsqueeze(1)
    xhat = _back(s["codes"], s["scales"]) * r
    g = s["grad"].float()
    wg = g * s["weight"].float()
    d = r * (wg - xhat * (wg * xhat).mean(1, keepdim=True))
    if case["residual"]:
        d = d + s["residual"].float()
    return {"grad_x": d.to(torch.bfloat16), "grad_weight": (g * xhat).sum(0)}


# ---- the package's operators -------------------------------------------------------------------


def _run_own(s):
    from nvfp4_block_scaled_quantize_gb300 import api
    case, op = s["case"], s["case"]["op"]
    if op == "plan":
        return api.nvfp4_moe_plan(s["ids"], case["experts"])
    if op == "dispatch":
        packed, amax = api.nvfp4_moe_dispatch(s["x"], s["plan"])
        return {"packed": packed, "amax": amax}
    if op == "dispatch_backward":
        return {"grad_x": api.nvfp4_moe_dispatch_backward(s["grad"], s["plan"])}
    if op == "combine":
        return {"out": api.nvfp4_moe_combine(s["y"], s["weights"], s["plan"])}
    if op == "combine_backward":
        gy, gw = api.nvfp4_moe_combine_backward(s["grad"], s["y"], s["weights"], s["plan"])
        return {"grad_y": gy, "grad_weights": gw}
    if op == "swiglu_checkpoint":
        out = api.nvfp4_swiglu_checkpoint(s["x"], offsets=s["offsets"])
        return dict(out, codes=out["codes"].view(torch.float8_e4m3fn))
    if op == "swiglu_checkpoint_backward":
        return {"grad_h": api.nvfp4_swiglu_checkpoint_backward(s["grad"], s["codes"], s["scales"],
                                                               offsets=s["offsets"])}
    if op == "rmsnorm_checkpoint":
        out = api.nvfp4_rmsnorm_checkpoint(s["x"], s["weight"], eps=EPS)
        return dict(out, codes=out["codes"].view(torch.float8_e4m3fn))
    gx, gw = api.nvfp4_rmsnorm_checkpoint_backward(s["grad"], s["codes"], s["scales"], s["rstd"],
                                                   s["weight"], grad_residual=s.get("residual"))
    return {"grad_x": gx, "grad_weight": gw}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- 64 bits -----------------------------------------------------------------------------------


def _e4m3_of(x):
    """The E4M3 values of `x` [M, N] over their block's scale, from the definition in binary64."""
    M, N = x.shape
    b = x.double().reshape(M, -1, 32)
    m, e = torch.frexp(b.abs().amax(2, keepdim=True) / 448)
    e = torch.where(m == 0.5, e - 1, e).clamp_min(-127).double()
    v = b / torch.exp2(e)
    step = torch.exp2(torch.frexp(v)[1].double().sub(1).clamp_min(-6) - 3)
    return (torch.round(v / step) * step).reshape(M, N)


def _value_of(codes, scales):
    v = codes.view(torch.float8_e4m3fn).double()
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return None  # whole numbers only
    if "tokens" in case:
        plan, K = s["plan"], case["topk"]
        live = int(plan["offsets"][-1])
        slots = plan["slot_of_row"][:live].long()
        token, n = slots // K, case["tokens"]
        if op == "dispatch":
            packed = torch.zeros(n * K, case["hidden"], dtype=torch.float64, device="cuda")
            packed[:live] = s["x"].double()[token]
            return {"packed": packed, "amax": None}
        w = s["weights"].double().reshape(-1)[slots].unsqueeze(1) if "weights" in s else 1.0
        if op != "combine_backward":
            rows = (s["grad"] if op == "dispatch_backward" else s["y"])[:live].double()
            total = torch.zeros(n, case["hidden"], dtype=torch.float64, device="cuda")
            total.index_add_(0, token, rows * w)
            return {"grad_x" if op == "dispatch_backward" else "out": total}
        g = s["grad"].double()[token]
        grad_y = torch.zeros(n * K, case["hidden"], dtype=torch.float64, device="cuda")
        grad_y[:live] = g * w
        grad_w = torch.zeros(n * K, dtype=torch.float64, device="cuda")
        grad_w[slots] = (g * s["y"][:live].double()).sum(1)
        return {"grad_y": grad_y, "grad_weights": grad_w.reshape(n, K)}
    M, N = case["rows"], case["width"]
    if op.startswith("swiglu"):
        live = int(s["offsets"][-1])
        if op == "swiglu_checkpoint":
            h = s["x"].double()
            h[live:] = 0
            gate, up = h.split(N, dim=1)
            return {"y": gate / (1 + torch.exp(-gate)) * up, "codes": _e4m3_of(h), "scales": None,
                    "amax": None}
        gate, up = _value_of(s["codes"], s["scales"]).split(N, dim=1)
        dy = s["grad"].double()
        t = 1 + torch.exp(-gate)
        slope = 1 / t + gate * torch.exp(-gate) / (t * t)
        d = torch.cat([dy * up * slope, dy * gate / t], dim=1)
        d[live:] = 0
        return {"grad_h": d}
    if op == "rmsnorm_checkpoint":
        x = s["x"].double()
        rstd = 1 / torch.sqrt((x * x).sum(1) / N + EPS)
        return {"y": x * rstd[:, None] * s["weight"].double(), "codes": _e4m3_of(s["x"]),
                "scales": None, "rstd": rstd, "amax": None}
    r = s["rstd"].double()[:, None]
    x = _value_of(s["codes"], s["scales"])
    dy = s["grad"].double()
    dn = dy * s["weight"].double()
    # d/dx of x * r(x): r dn - r^3 x (x . dn) / N
    d = r * dn - r ** 3 * x * ((x * dn).sum(1, keepdim=True) / N)
    if case["residual"]:
        d = d + s["residual"].double()
    return {"grad_x": d, "grad_weight": (dy * x * r).sum(0)}
