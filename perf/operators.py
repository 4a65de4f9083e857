"""Workloads of the operators around the block-FP8 products: quant_norm, linear_w8a8_epilogue,
expert_plan and linear_w8a8_experts.

Each case is one call as a serving program makes it.  ``run`` computes it in elementary torch
operations (``own`` false) or through the library (``own`` true); ``exact`` computes the
definition in 64 bits.  Sizes follow the repository's projections (5120 x 5120, 17408 x 5120,
5000 x 4000, 7168-wide prefill) and generic expert layers.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 128
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------- cases

def _norm(name, M, K, kind="rms", x="bf16", h="bf16", post=False, gate="none", top=0, codes=True, plain="none"):
    return dict(name=name, op="norm", M=M, K=K, kind=kind, x=x, h=h, post=post, gate=gate, top=top, codes=codes,
                plain=plain)


def _epilogue(name, M, N, K, act, bias=True, residual=False, y="bf16"):
    return dict(name=name, op="epilogue", M=M, N=N, K=K, act=act, bias=bias, residual=residual, y=y)


def _experts(name, M, top, E, N, K, gather, y="bf16", skew=1.0):
    return dict(name=name, op="experts", M=M, top=top, E=E, N=N, K=K, gather=gather, y=y, skew=skew)


def _plan(name, M, top, E, drop=False):
    return dict(name=name, op="plan", M=M, top=top, E=E, drop=drop)


def listed():
    return [
        # one decoded token between two blocks: residual add, RMS norm, codes for the next projection
        _norm("norm-decode-1x5120", 1, 5120),
        # prefill of a sandwich-norm model: norm after the block, per-channel gate, residual, norm before the next
        _norm("norm-post-gate-8192x7168", 8192, 7168, post=True, gate="row"),
        # layer norm with biases, per-token modulation, float32 stream, a width that ends inside a scale group;
        # the router reads the unquantized norm beside the codes
        _norm("norm-layer-333x5000-f32", 333, 5000, kind="layer", x="f32", h="f32", post=True, gate="token", plain="f32"),
        # the experts' outputs of 1024 tokens summed by router weight into the stream, then the next norm
        _norm("norm-combine8-1024x4096", 1024, 4096, top=8, plain="bf16"),
        # output projection of one decoded token: bias and residual in the product
        _epilogue("epilogue-decode-1x5120x5120", 1, 5120, 5120, "none", residual=True),
        # FFN up projection of 1024 prompt tokens with bias and tanh GELU
        _epilogue("epilogue-gelu-1024x17408x5120", 1024, 17408, 5120, "gelu_tanh"),
        # odd sizes, float32 output and stream, SiLU
        _epilogue("epilogue-silu-333x5000x4000-f32", 333, 5000, 4000, "silu", residual=True, y="f32"),
        # one decoded token over 8 of 64 experts: gate/up
        _experts("experts-decode-1x8of64", 1, 8, 64, 1536, 2048, True),
        # a decode batch over 4 of 32 experts: down projection of rows already in expert order
        _experts("experts-batch-48x4of32", 48, 4, 32, 2048, 1408, False, y="f32"),
        # prefill over 4 of 32 experts: gate/up
        _experts("experts-prefill-4096x4of32", 4096, 4, 32, 2816, 2048, True),
        # router choices of a decode batch
        _plan("plan-64x8of64", 64, 8, 64),
        # router choices of a large prefill, some dropped by a capacity rule
        _plan("plan-8192x8of128", 8192, 8, 128, drop=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "epilogue", "experts", "plan"])
    if op == "norm":
        K = _log(rng, 300, 8192)
        top = rng.choice([0, 0, 2, 4])
        M = max(1, _log(rng, 1, 4 * 10 ** 7 // (K * max(1, top))))
        c = _norm("", M, K, rng.choice(["rms", "layer"]), rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32"]),
                  rng.choice([True, False]), rng.choice(["none", "row", "token"]), top, True,
                  rng.choice(["none", "none", "bf16", "f32"]))
    elif op == "epilogue":
        N, K = _log(rng, 400, 17408), _log(rng, 400, 5120)
        if rng.random() < 0.75:
            K = max(16, K // 16 * 16)
        M = _log(rng, 1, 1024)
        c = _epilogue("", M, N, K, rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]), rng.choice([True, False]),
                      rng.choice([True, False]), rng.choice(["bf16", "f32"]))
    elif op == "experts":
        N, K = _log(rng, 300, 2816), _log(rng, 300, 2048)
        if rng.random() < 0.75:
            K = max(16, K // 16 * 16)
        E = _log(rng, 2, min(96, 18 * 10 ** 7 // (N * K)))
        top = min(E, rng.choice([1, 2, 4, 6, 8]))
        c = _experts("", _log(rng, 1, 16000 // top), top, E, N, K, rng.choice([True, False]),
                     rng.choice(["bf16", "f32"]), rng.choice([0.0, 1.0, 2.0]))
    else:
        E = _log(rng, 2, 256)
        c = _plan("", _log(rng, 1, 8192), min(E, rng.choice([1, 2, 4, 6, 8])), E, rng.choice([True, False]))
    del c["name"]
    return c


# ------------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activations(g, M, K):
    """Normal values with one channel in a hundred 20 times larger, as transformer streams have them."""
    gain = torch.where(torch.rand(K, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    return _randn(g, M, K) * gain


def _e4m3(v):
    return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _groups(v):
    """The last axis in groups of 128, zero-filled."""
    K = v.shape[-1]
    return torch.nn.functional.pad(v, (0, -K % BLOCK)).unflatten(-1, (-1, BLOCK))


def _quantize(n):
    """Float32 rows -> (E4M3 values [M, K], scales [M, ceil(K/128)])."""
    K = n.shape[-1]
    v = _groups(n)
    s = v.abs().amax(-1).clamp(min=1e-10) / 448.0
    return _e4m3(v / s[..., None]).flatten(-2)[..., :K].contiguous(), s


def _weights(g, E, N, K):
    """E weights [N, K] as a converter stores them: E4M3 codes and bfloat16 scales per 128 x 128 block."""
    codes = torch.empty(E, N, K, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, -(-N // BLOCK), -(-K // BLOCK), dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        w = _randn(g, N, K) * 0.02
        t = torch.nn.functional.pad(w, (0, -K % BLOCK, 0, -N % BLOCK))
        t = t.unflatten(1, (-1, BLOCK)).unflatten(0, (-1, BLOCK))
        s = (t.abs().amax((1, 3)) / 448.0).to(torch.bfloat16)
        scales[e] = s
        q = _e4m3(t / s.float()[:, None, :, None])
        codes[e] = q.flatten(2, 3).flatten(0, 1)[:N, :K].view(torch.uint8)
    return codes, scales


def _choices(g, M, top, E, skew):
    """The router's choices: ``top`` different experts a token, some experts preferred by ``skew``."""
    logits = _randn(g, M, E) + skew * _randn(g, E)
    p, ids = logits.topk(top, -1)
    return ids.to(torch.int32), torch.softmax(p, -1)


def _sorted_rows(ids, E):
    """(offsets, rows, slots) of the choices, stable by expert; ids outside [0, E) have no slot."""
    M, top = ids.shape
    flat = ids.flatten().long()
    ok = (flat >= 0) & (flat < E)
    key, order = torch.sort(torch.where(ok, flat, E), stable=True)
    bounds = torch.arange(E + 1, device=ids.device)
    offsets = torch.searchsorted(key, bounds).int()
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=ids.device)
    slots = torch.where(ok, place, -1).int().view(M, top)
    rows = torch.where(key < E, order // top, -1).int()
    return offsets, rows, slots


def _weight_vector(g, K, near):
    return (near + 0.1 * _randn(g, K)).to(torch.bfloat16)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "norm":
        M, K, top = case["M"], case["K"], case["top"]
        R = M * max(1, top)
        s["rows_in"] = _activations(g, R, K).to(DT[case["x"]])
        s["residual"] = (2.0 * _activations(g, M, K)).to(DT[case["h"]])
        s["weight"] = _weight_vector(g, K, 1.0)
        s["bias"] = _weight_vector(g, K, 0.0) if case["kind"] == "layer" else None
        s["post_weight"] = _weight_vector(g, K, 1.0) if case["post"] else None
        s["post_bias"] = _weight_vector(g, K, 0.0) if case["post"] and case["kind"] == "layer" else None
        s["gate"] = {"none": None, "row": _weight_vector(g, K, 0.5)}.get(case["gate"])
        if case["gate"] == "token":
            s["gate"] = (0.5 + 0.1 * _randn(g, M, K)).to(torch.bfloat16)
        s["slots"] = s["probs"] = None
        if top:
            s["slots"] = torch.randperm(R, generator=g, device="cuda").int().view(M, top)
            s["probs"] = torch.softmax(_randn(g, M, top), -1)
    elif case["op"] == "epilogue":
        M, N, K = case["M"], case["N"], case["K"]
        codes, scales = _weights(g, 1, N, K)
        s["codes"], s["scales"] = codes[0], scales[0]
        q, s["xs"] = _quantize(_activations(g, M, K))
        s["xq"] = q.view(torch.uint8)
        s["bias"] = (0.1 * _randn(g, N)).to(torch.bfloat16) if case["bias"] else None
        s["residual"] = _activations(g, M, N).to(DT[case["y"]]) if case["residual"] else None
        if own:
            import block_scaled_fp8_linear_amd as B
            s["handle"] = B.BlockFP8Weight([(s["codes"], s["scales"])])
    elif case["op"] == "experts":
        M, top, E, N, K = (case[k] for k in ("M", "top", "E", "N", "K"))
        s["codes"], s["scales"] = _weights(g, E, N, K)
        ids, _ = _choices(g, M, top, E, case["skew"])
        s["offsets"], rows, _ = _sorted_rows(ids, E)
        s["rows"] = rows if case["gather"] else None
        q, s["xs"] = _quantize(_activations(g, M if case["gather"] else M * top, K))
        s["xq"] = q.view(torch.uint8)
        # the plain form slices by host numbers, which such a program keeps
        s["ends"] = s["offsets"].tolist()
        if own:
            import block_scaled_fp8_linear_amd as B
            s["handle"] = B.ExpertsFP8Weight([(s["codes"], s["scales"])])
    else:
        s["ids"], _ = _choices(g, case["M"], case["top"], case["E"], 1.0)
        if case["drop"]:
            lost = torch.rand(s["ids"].shape, generator=g, device="cuda") < 0.05
            s["ids"] = torch.where(lost, -1, s["ids"])
        # rows behind the last expert's keep what they hold
        s["rows"] = torch.full((case["M"] * case["top"],), -1, dtype=torch.int32, device="cuda")
    return s


# --------------------------------------------------------------------------------- plain form

def _normed(v, kind, eps, weight, bias):
    """Norm of float64 rows; 64 bits because the codes that follow are values next to a border."""
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    v = v * (1.0 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)) * weight.double()
    return v if bias is None else v + bias.double()


def _plain_norm(s):
    x = s["rows_in"].double()
    if s["top"]:
        x = (x[s["slots"].long()] * s["probs"].double()[..., None]).sum(1)
    if s["post"]:
        x = _normed(x, s["kind"], 1e-6, s["post_weight"], s["post_bias"])
    if s["gate"] is not None:
        x = x * s["gate"].double()
    h = (0.5 * s["residual"].double() + x).float().to(DT[s["h"]])
    n = _normed(h.double(), s["kind"], 1e-6, s["weight"], s["bias"]).float()
    q, xs = _quantize(n)
    return [q, xs, h] + ([n.to(DT[s["plain"]])] if s["plain"] != "none" else [])


def _weight_f32(codes, scales):
    """Float32 weight: the E4M3 values times their block's scale."""
    N, K = codes.shape
    per = scales.float().repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
    return codes.view(torch.float8_e4m3fn).float() * per


def _rows_f32(xq, xs):
    return xq.view(torch.float8_e4m3fn).float() * xs.repeat_interleave(BLOCK, 1)[:, :xq.shape[1]]


def _act(v, act):
    if act == "relu":
        return v.clamp(min=0.0)
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _plain_epilogue(s):
    y = _rows_f32(s["xq"], s["xs"]) @ _weight_f32(s["codes"], s["scales"]).t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = _act(y, s["act"])
    if s["residual"] is not None:
        y = y + 0.5 * s["residual"].float()
    return y.to(DT[s["y"]])


def _plain_experts(s):
    x = _rows_f32(s["xq"], s["xs"])
    if s["rows"] is not None:
        x = x[s["rows"].long()]
    E, ends = s["E"], s["ends"]
    if x.shape[0] <= E:
        # fewer rows than experts: each row with its expert's weight
        e = torch.searchsorted(s["offsets"], torch.arange(x.shape[0], device=x.device, dtype=torch.int32), right=True) - 1
        w = s["codes"][e].view(torch.float8_e4m3fn).float()
        per = s["scales"][e].float().repeat_interleave(BLOCK, 1)[:, :s["N"]].repeat_interleave(BLOCK, 2)[:, :, :s["K"]]
        return ((w * per) @ x[:, :, None])[:, :, 0].to(DT[s["y"]])
    # one product an expert: padding them to one size would multiply the largest expert's rows by E
    y = [x[ends[e]:ends[e + 1]] @ _weight_f32(s["codes"][e], s["scales"][e]).t() for e in range(E) if ends[e + 1] > ends[e]]
    return torch.cat(y).to(DT[s["y"]])


def _plain_plan(s):
    return list(_sorted_rows(s["ids"], s["E"]))


# --------------------------------------------------------------------------------------- run

def run(s):
    if not own:
        return {"norm": _plain_norm, "epilogue": _plain_epilogue, "experts": _plain_experts, "plan": _plain_plan}[s["op"]](s)
    import block_scaled_fp8_linear_amd as B
    if s["op"] == "norm":
        xq, xs, h, n = B.quant_norm(s["rows_in"], s["weight"], bias=s["bias"], kind=s["kind"], eps=1e-6,
                                    residual=s["residual"], residual_scale=0.5, gate=s["gate"],
                                    post_weight=s["post_weight"], post_bias=s["post_bias"], slots=s["slots"],
                                    probs=s["probs"], out_dtype=DT.get(s["plain"]))
        return [xq.view(torch.float8_e4m3fn), xs, h] + ([n] if n is not None else [])
    if s["op"] == "epilogue":
        return B.linear_w8a8_epilogue(s["handle"], s["xq"], s["xs"], bias=s["bias"], activation=s["act"],
                                      residual=s["residual"], residual_scale=0.5, out_dtype=DT[s["y"]])
    if s["op"] == "experts":
        return B.linear_w8a8_experts(s["handle"], s["xq"], s["xs"], s["offsets"], rows=s["rows"], out_dtype=DT[s["y"]])
    return list(B.expert_plan(s["ids"], s["E"], rows=s["rows"]))


# -------------------------------------------------------------------------------------- work

def work(case):
    if case["op"] == "norm":
        M, K, top = case["M"], case["K"], case["top"]
        b = M * K * ((2 if case["x"] == "bf16" else 4) * max(1, top) + 2 * (2 if case["h"] == "bf16" else 4) + 1)
        b += 4 * M * -(-K // BLOCK) + 8 * M * top
        b += {"none": 0, "bf16": 2, "f32": 4}[case["plain"]] * M * K
        b += 2 * K * (1 + (1 + case["post"]) * (case["kind"] == "layer") + case["post"] + (case["gate"] == "row"))
        b += 2 * M * K * (case["gate"] == "token")
        return {"bytes": b, "flops": M * K * (10 + 2 * top + 6 * case["post"])}
    if case["op"] == "epilogue":
        M, N, K = case["M"], case["N"], case["K"]
        y = 2 if case["y"] == "bf16" else 4
        b = N * K + M * K + 4 * M * -(-K // BLOCK) + 2 * -(-N // BLOCK) * -(-K // BLOCK)
        b += y * M * N * (1 + case["residual"]) + 2 * N * case["bias"]
        return {"bytes": b, "flops": 2 * M * N * K}
    if case["op"] == "experts":
        M, top, E, N, K = (case[k] for k in ("M", "top", "E", "N", "K"))
        R = M * top
        # experts that have rows: every token takes ``top`` different ones of E
        used = E * (1.0 - (1.0 - top / E) ** M)
        b = used * (N * K + 2 * -(-N // BLOCK) * -(-K // BLOCK))
        b += (M if case["gather"] else R) * (K + 4 * -(-K // BLOCK)) + 4 * R * case["gather"] + 4 * (E + 1)
        b += (2 if case["y"] == "bf16" else 4) * R * N
        return {"bytes": b, "flops": 2 * R * N * K}
    return {"bytes": 12 * case["M"] * case["top"] + 4 * (case["E"] + 1), "flops": 0}


# ------------------------------------------------------------------------------------- exact

def _nearest_e4m3(v):
    """E4M3 values of float64 values: nearest, ties to even, saturating at 448."""
    a = v.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))).clamp(min=-6.0) - 3.0)
    return torch.copysign((torch.round(a / step) * step).clamp(max=448.0), v)


def _exact_stats(v, kind):
    mu = v.sum(-1, keepdim=True) / v.shape[-1] if kind == "layer" else torch.zeros_like(v[..., :1])
    return mu, ((v - mu) ** 2).sum(-1, keepdim=True) / v.shape[-1]


def _exact_norm(s):
    M, K = s["M"], s["K"]
    o = s["rows_in"].to(torch.float64)
    if s["top"]:
        total = torch.zeros(M, K, dtype=torch.float64, device=o.device)
        for j in range(s["top"]):
            total += s["probs"][:, j, None].to(torch.float64) * o.index_select(0, s["slots"][:, j].long())
        o = total
    if s["post_weight"] is not None:
        mu, var = _exact_stats(o, s["kind"])
        o = (o - mu) / torch.sqrt(var + 1e-6) * s["post_weight"].to(torch.float64)
        o = o + s["post_bias"].to(torch.float64) if s["post_bias"] is not None else o
    if s["gate"] is not None:
        o = o * s["gate"].to(torch.float64)
    h = s["residual"].to(torch.float64) / 2 + o
    # the norm reads the stream as it is stored
    kept = h.to(torch.float32).to(s["residual"].dtype).to(torch.float64)
    mu, var = _exact_stats(kept, s["kind"])
    n = (kept - mu) / torch.sqrt(var + 1e-6) * s["weight"].to(torch.float64)
    n = n + s["bias"].to(torch.float64) if s["bias"] is not None else n
    Kb = -(-K // BLOCK)
    wide = torch.zeros(M, Kb * BLOCK, dtype=torch.float64, device=n.device)
    wide[:, :K] = n
    wide = wide.view(M, Kb, BLOCK)
    scale = torch.clamp(wide.abs().max(-1).values, min=1e-10) / 448
    # codes are defined on the float32 values of the norm and its scale
    near = wide.float()
    near = near / (torch.clamp(near.abs().max(-1, keepdim=True).values, min=1e-10) / 448)
    q = _nearest_e4m3(near.to(torch.float64)).view(M, -1)[:, :K]
    return [q, scale, h] + ([n] if s["plain"] != "none" else [])


def _exact_scaled(codes, scales, rows_per_scale):
    v = codes.view(torch.float8_e4m3fn).to(torch.float64)
    r = torch.arange(v.shape[0], device=v.device) // rows_per_scale
    c = torch.arange(v.shape[1], device=v.device) // BLOCK
    return v * scales.to(torch.float64)[r[:, None], c[None, :]]


def _exact_epilogue(s):
    z = _exact_scaled(s["xq"], s["xs"], 1).matmul(_exact_scaled(s["codes"], s["scales"], BLOCK).t())
    if s["bias"] is not None:
        z += s["bias"].to(torch.float64)
    a = s["act"]
    if a == "relu":
        z = torch.where(z > 0, z, torch.zeros_like(z))
    elif a == "silu":
        z = z * torch.sigmoid(z)
    elif a == "gelu":
        z = z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
    elif a == "gelu_tanh":
        z = z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    return z if s["residual"] is None else z + s["residual"].to(torch.float64) / 2


def _exact_experts(s):
    x = _exact_scaled(s["xq"], s["xs"], 1)
    R = s["M"] * s["top"]
    y = torch.zeros(R, s["N"], dtype=torch.float64, device=x.device)
    at = s["offsets"].cpu().numpy()
    for e in range(s["E"]):
        mine = torch.arange(int(at[e]), int(at[e + 1]), device=x.device)
        if mine.numel():
            of = mine if s["rows"] is None else s["rows"][mine].long()
            y[mine] = x[of].matmul(_exact_scaled(s["codes"][e], s["scales"][e], BLOCK).t())
    return y


def exact(case, seed):
    """Whole numbers have no nearer value: expert_plan has None here."""
    s = prepare(case, seed)
    f = {"norm": _exact_norm, "epilogue": _exact_epilogue, "experts": _exact_experts}.get(case["op"])
    return None if f is None else f(s)
