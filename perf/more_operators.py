"""Workloads of the operators between the Q/K/V projection and the output projection: rope, cache_write, cache_read and
paged_attention.

Each case is one call as a serving program makes it.  ``run`` computes it in elementary torch operations (``own`` false) or
through the library (``own`` true); ``exact`` computes the definition in 64 bits.  Sizes follow the repository's projections
(queries of 5120 and 6144 features) and generic head layouts.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 128
EPS = 1e-6
DT = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.uint8}
SIZE = {"bf16": 2, "f32": 4, "e4m3": 1}


# ------------------------------------------------------------------------------------- cases

def _rope(name, M, heads, kv, D, R, axes=1, order="blocks", pairing="half", x="bf16", y="bf16", norm=False):
    return dict(name=name, op="rope", M=M, heads=heads, kv=kv, D=D, R=R, axes=axes, order=order, pairing=pairing, x=x,
                y=y, norm=norm)


def _write(name, M, kv, D, page, cache="e4m3", x="bf16", R=0, heads=0, norm=False, pairing="half", drop=False):
    return dict(name=name, op="write", M=M, kv=kv, D=D, page=page, cache=cache, x=x, R=R, heads=heads, norm=norm,
                pairing=pairing, drop=drop)


def _read(name, B, longest, kv, D, page, cache="e4m3", y="bf16"):
    return dict(name=name, op="read", B=B, longest=longest, kv=kv, D=D, page=page, cache=cache, y=y)


def _attention(name, B, longest, heads, kv, D, page, cache="bf16", q="bf16", window=0, lse=False, empty=False):
    return dict(name=name, op="attention", B=B, longest=longest, heads=heads, kv=kv, D=D, page=page, cache=cache, q=q,
                window=window, lse=lse, empty=empty)


def listed():
    return [
        # one decoded token: queries and keys of a 5120-wide model, text positions far into a long prompt
        _rope("rope-decode-1x40+8x128", 1, 40, 8, 128, 128),
        # a video prompt: time, height and width in blocks of the pairs, from a float32 projection
        _rope("rope-video-4096x40+8x128", 4096, 40, 8, 128, 128, axes=3, x="f32"),
        # a decode batch: head norms, a quarter of the channels rotated, queries in the same call, codes into the cache
        _write("write-decode-48x24+4x256", 48, 4, 256, 16, R=64, heads=24, norm=True),
        # a prompt's keys (rotated on the way) and values as codes
        _write("write-prefill-8192x8x128", 8192, 8, 128, 64, R=128),
        # odd sizes: bfloat16 cache, float32 projection, neighbouring channels paired, padded tokens dropped
        _write("write-333x3x80-bf16", 333, 3, 80, 24, cache="bf16", x="f32", R=80, pairing="adjacent", drop=True),
        # the cached prefixes of eight prompts for a dense prefill attention
        _read("read-prefix-8x4096x8x128", 8, 4096, 8, 128, 64),
        # many short ragged prefixes of a bfloat16 cache with odd pages, to float32
        _read("read-ragged-37x700x5x96-f32", 37, 700, 5, 96, 24, cache="bf16", y="f32"),
        # one user, a short chat
        _attention("attention-1x1000-40of8x128", 1, 1000, 40, 8, 128, 16),
        # one user, a very long document, codes
        _attention("attention-1x131072-32of4x128", 1, 131072, 32, 4, 128, 64, cache="e4m3"),
        # a full serving batch of ragged lengths, codes
        _attention("attention-64x8192-40of8x128", 64, 8192, 40, 8, 128, 16, cache="e4m3"),
        # odd sizes: float32 queries, wide heads, pages of 24, a sliding window, a padded row, log-sum-exp asked for
        _attention("attention-7x5000-24of4x256", 7, 5000, 24, 4, 256, 24, q="f32", window=2048, lse=True, empty=True),
        # many short chats, a key head for each query head
        _attention("attention-256x1000-24of24x80", 256, 1000, 24, 24, 80, 32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attention", "attention"])
    D = rng.choice([64, 80, 96, 128, 128, 192, 256])
    page = rng.choice([1, 7, 16, 16, 24, 32, 64, 128, 256])
    cache = rng.choice(["bf16", "e4m3"])
    if op == "rope":
        R = rng.choice([D, D, D // 2, D // 4 // 2 * 2])
        heads, kv = rng.choice([1, 8, 24, 40, 64]), rng.choice([0, 1, 3, 8])
        axes = rng.choice([1, 1, 2, 3, 4])
        c = _rope("", _log(rng, 1, max(1, 4096 * 48 * 128 // ((heads + kv) * D))), heads, kv, D, R, axes,
                  rng.choice(["blocks", "turns"]), rng.choice(["half", "adjacent"]), rng.choice(["bf16", "f32"]),
                  rng.choice(["bf16", "f32"]), rng.choice([True, False]))
    elif op == "write":
        kv, heads = rng.choice([1, 3, 4, 8, 16]), rng.choice([0, 0, 8, 24, 40])
        M = _log(rng, 1, max(1, 8192 * 16 * 128 // ((2 * kv + heads) * D)))
        c = _write("", M, kv, D, page, cache, rng.choice(["bf16", "f32"]), 0 if heads == 0 and rng.random() < 0.3 else D // rng.choice([1, 2, 4]) // 2 * 2,
                   heads, rng.choice([True, False]), rng.choice(["half", "adjacent"]), rng.choice([True, False]))
        c["norm"] = c["norm"] and c["R"] > 0
    elif op == "read":
        kv = rng.choice([1, 3, 4, 8, 16])
        longest = _log(rng, 1, 8192)
        B = _log(rng, 1, max(1, min(128, 8 * 4096 * 8 * 128 // (longest * kv * D))))
        c = _read("", B, longest, kv, D, page, cache, rng.choice(["bf16", "f32"]))
    else:
        kv, G = rng.choice([1, 2, 4, 8, 24]), rng.choice([1, 2, 4, 5, 8, 16, 20])
        longest = _log(rng, 1, 65536)
        B = _log(rng, 1, max(1, min(256, 300 * 10 ** 6 // (longest * kv * max(G, 2) * D))))
        c = _attention("", B, longest, kv * G, kv, D, page, cache, rng.choice(["bf16", "bf16", "f32"]),
                       rng.choice([0, 0, 0, _log(rng, 1, longest)]), rng.choice([True, False]), B > 1 and rng.choice([True, False]))
    del c["name"]
    return c


# ------------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _lengths(case):
    """Lengths from short to the longest, most of them short, as a batch that is being served has them; one is empty where
    the case says so."""
    B, longest = case["B"], case["longest"]
    n = [max(1, round(longest * ((i + 1) / B) ** 2)) for i in range(B)]
    if case.get("empty"):
        n[0] = 0
    return n


def _projected(g, M, heads, D, x):
    """Heads of a projection's output: some channels much larger than others, as keys have them."""
    gain = torch.exp(0.5 * _randn(g, heads, D))
    return (_randn(g, M, heads, D) * gain).to(DT[x])


def _codes(v):
    """Float32 [..., D] -> (E4M3 codes, scales [..., ceil(D/128)]), the activation quantizer's format."""
    D = v.shape[-1]
    t = torch.nn.functional.pad(v, (0, -D % BLOCK)).unflatten(-1, (-1, BLOCK))
    amax = t.abs().amax(-1).clamp(min=1e-10)
    # (a tensor of 448: torch divides by a number as a product with its rounded reciprocal)
    scale = amax / torch.full_like(amax, 448.0)
    q = (t / scale[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.flatten(-2)[..., :D].contiguous().view(torch.uint8), scale


def _cache(g, case, pages):
    """A paged cache that holds values: head-major pages, seen as [pages, page, heads, D]; scales [pages, page, heads, groups]
    with the page's tokens next to each other."""
    kv, D, page = case["kv"], case["D"], case["page"]
    out = {}
    for which in ("k", "v"):
        t = torch.empty(pages, kv, page, D, dtype=DT[case["cache"]], device="cuda")
        sc = torch.empty(pages, kv, -(-D // BLOCK), page, dtype=torch.float32, device="cuda") if case["cache"] == "e4m3" else None
        gain = torch.exp(0.5 * _randn(g, kv, 1, D))
        step = max(1, (1 << 26) // (kv * page * D))
        for p in range(0, pages, step):   # in parts: the float32 values would take four times the cache
            part = _randn(g, min(step, pages - p), kv, page, D) * gain
            if sc is None:
                t[p:p + step] = part.to(torch.bfloat16)
            else:
                q, s = _codes(part)
                t[p:p + step] = q
                sc[p:p + step] = s.transpose(2, 3)
        out[which] = t.transpose(1, 2)
        out[which + "_scale"] = None if sc is None else sc.permute(0, 3, 1, 2)
    return out


def _handle(s):
    import block_scaled_fp8_linear_amd as B
    return B.PagedKVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])


def _sections(case):
    """Pairs of each axis: the first takes what the others leave."""
    n, a = case["R"] // 2, case["axes"]
    rest = [n // a] * (a - 1)
    return [n - sum(rest)] + rest


def _axis_of_pair(case):
    """The axis of each pair: in blocks, or in turns as far as each axis's pairs go (then the first)."""
    sec = _sections(case)
    if case["order"] == "blocks":
        return [a for a, n in enumerate(sec) for _ in range(n)]
    A = len(sec)
    return [i % A if i < A * sec[i % A] else 0 for i in range(case["R"] // 2)]


def _rotation(g, s, case):
    """What a model keeps for its rotary positions, and the tokens' positions."""
    R, M, axes = case["R"], case["M"], case.get("axes", 1)
    s["inv_freq"] = s["positions"] = s["q_weight"] = s["k_weight"] = None
    if R:
        s["inv_freq"] = (1e6 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)).float()
        first = torch.randint(0, 120000, (axes, 1), generator=g, device="cuda")
        along = torch.arange(M, device="cuda")
        rows = [along, along // 7 % 60, along % 7, along % 3][:axes]
        p = first + torch.stack(rows)
        s["positions"] = (p[0] if axes == 1 else p).to(torch.int32)
    if case["norm"]:
        for w in ("q_weight", "k_weight"):
            s[w] = (1.0 + 0.1 * _randn(g, case["D"])).to(torch.bfloat16)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    D, kv = case["D"], case["kv"]
    if case["op"] == "rope":
        x = _projected(g, case["M"], case["heads"] + 2 * kv, D, case["x"])
        # queries and keys as the grouped projection leaves them: next to each other and to the values
        s["q"] = x[:, :case["heads"]]
        s["k"] = x[:, case["heads"]:case["heads"] + kv] if kv else None
        _rotation(g, s, case)
        s["axis"] = _axis_of_pair(case)
        s["axis_dev"] = torch.tensor(s["axis"], device="cuda")
        if own:
            import block_scaled_fp8_linear_amd as B
            s["axes_handle"] = B.rope_axes(_sections(case), interleaved=case["order"] == "turns") if case["axes"] > 1 else None
    elif case["op"] == "write":
        M, heads, page = case["M"], case["heads"], case["page"]
        x = _projected(g, M, heads + 2 * kv, D, case["x"])
        s["q"] = x[:, :heads] if heads else None
        s["kx"], s["vx"] = x[:, heads:heads + kv], x[:, heads + kv:]
        pages = -(-M // page) + 2
        s.update(_cache(g, case, pages))
        s["slots"] = torch.randperm(pages * page, generator=g, device="cuda")[:M].contiguous()
        if case["drop"]:
            s["slots"] = torch.where(torch.rand(M, generator=g, device="cuda") < 0.1, -1, s["slots"])
        # the plain form picks the kept tokens by their numbers, which such a program has
        s["kept"] = (s["slots"] >= 0).nonzero()[:, 0]
        _rotation(g, s, case)
        if own:
            s["handle"] = _handle(s)
    else:
        B, page = case["B"], case["page"]
        n = _lengths(case)
        order = torch.randperm(B, generator=g, device="cuda").tolist()
        n = [n[i] for i in order]
        need = [-(-v // page) for v in n]
        pages = sum(need) + 3
        s.update(_cache(g, case, pages))
        # pages of a sequence lie anywhere; entries behind its last page name none
        perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((B, max(1, max(need))), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b in range(B):
            table[b, :need[b]] = perm[at:at + need[b]]
            at += need[b]
        s["table"], s["n"] = table, n   # the plain form slices by host numbers, which such a program keeps
        if case["op"] == "read":
            ends = [0]
            for v in n:
                ends.append(ends[-1] + v)
            s["rows"] = ends[-1]
            s["offsets"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
        else:
            s["lens"] = torch.tensor(n, dtype=torch.int32, device="cuda")
            s["q"] = (2.0 * _randn(g, B, case["heads"], D)).to(DT[case["q"]])
        if own:
            s["handle"] = _handle(s)
    return s


# --------------------------------------------------------------------------------- plain form

def _turn(x, s, weight):
    """Head norm and rotation of x [M, H, D] in float64 (angles of far positions, and codes that lie next to a border),
    rounded to float32."""
    v = x.double()
    D, R = v.shape[-1], s["R"]
    if weight is not None:
        v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS) * weight.double()
    if R:
        p = s["positions"].double()
        if p.dim() == 2:
            p = p[s["axis_dev"]].t()          # [M, R/2]: each pair with its axis's position
        else:
            p = p[:, None]
        angle = p * s["inv_freq"].double()
        c, sn = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
        if s["pairing"] == "half":
            a, b, rest = v[..., :R // 2], v[..., R // 2:R], v[..., R:]
            v = torch.cat([a * c - b * sn, b * c + a * sn, rest], -1)
        else:
            a, b, rest = v[..., 0:R:2], v[..., 1:R:2], v[..., R:]
            v = torch.cat([torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2), rest], -1)
    return v.float()


def _plain_rope(s):
    y = DT[s["y"]]
    out = [_turn(s["q"], s, s["q_weight"]).to(y)]
    return out + ([_turn(s["k"], s, s["k_weight"]).to(y)] if s["k"] is not None else [])


def _held(t):
    """A cache's tensor as the values its codes stand for."""
    return t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t


def _plain_write(s):
    slot = s["slots"][s["kept"]]
    page, row = slot // s["page"], slot % s["page"]
    for x, name, weight in ((_turn(s["kx"], s, s["k_weight"]), "k", True), (s["vx"].float(), "v", False)):
        x = x[s["kept"]]
        if s["cache"] == "e4m3":
            q, scale = _codes(x)
            s[name][page, row] = q
            s[name + "_scale"][page, row] = scale
        else:
            s[name][page, row] = x.to(torch.bfloat16)
    out = [_held(s["k"]), _held(s["v"])]
    if s["cache"] == "e4m3":
        out += [s["k_scale"], s["v_scale"]]
    if s["q"] is not None:
        out.append(_turn(s["q"], s, s["q_weight"]).to(s["q"].dtype))
    return out


def _sequence(s, which, b, first, last):
    """Float32 rows [last - first, heads, D] of sequence b's positions first .. last - 1."""
    page = s["page"]
    p0 = first // page
    pages = s["table"][b, p0:-(-last // page)].long()
    t = _held(s[which])[pages].float()
    if s["cache"] == "e4m3":
        t = t * s[which + "_scale"][pages].repeat_interleave(BLOCK, -1)[..., :s["D"]]
    return t.flatten(0, 1)[first - p0 * page:last - p0 * page]


def _plain_read(s):
    y = DT[s["y"]]
    return [torch.cat([_sequence(s, which, b, 0, n) for b, n in enumerate(s["n"])]).to(y) for which in ("k", "v")]


def _span(s, n):
    return max(0, n - s["window"]) if s["window"] else 0


def _plain_attention(s):
    B, H, kv, D = len(s["n"]), s["heads"], s["kv"], s["D"]
    q = s["q"].float().view(B, kv, H // kv, D) * (D ** -0.5)
    out = torch.zeros(B, kv, H // kv, D, device=q.device)
    lse = torch.full((B, kv, H // kv), -math.inf, device=q.device)
    for b, n in enumerate(s["n"]):
        if n == 0:
            continue
        k, v = _sequence(s, "k", b, _span(s, n), n), _sequence(s, "v", b, _span(s, n), n)
        logits = q[b] @ k.permute(1, 2, 0).contiguous()
        m = logits.amax(-1, keepdim=True)
        p = torch.exp(logits - m)
        total = p.sum(-1, keepdim=True)
        out[b] = p @ v.transpose(0, 1).contiguous() / total
        lse[b] = (m + torch.log(total))[..., 0]
    out = out.view(B, H, D).to(s["q"].dtype)
    return [out, lse.view(B, H)] if s["lse"] else out


# --------------------------------------------------------------------------------------- run

def run(s):
    if not own:
        return {"rope": _plain_rope, "write": _plain_write, "read": _plain_read, "attention": _plain_attention}[s["op"]](s)
    import block_scaled_fp8_linear_amd as B
    if s["op"] == "rope":
        q, k = B.rope(s["q"], s["positions"], s["inv_freq"], k=s["k"], axes=s["axes_handle"], pairing=s["pairing"],
                      q_weight=s["q_weight"], k_weight=s["k_weight"] if s["k"] is not None else None, eps=EPS,
                      out_dtype=DT[s["y"]])
        return [q] if k is None else [q, k]
    if s["op"] == "write":
        q = B.cache_write(s["handle"], s["kx"], s["vx"], s["slots"], positions=s["positions"], inv_freq=s["inv_freq"],
                          pairing=s["pairing"], k_weight=s["k_weight"], q=s["q"],
                          q_weight=s["q_weight"] if s["q"] is not None else None, eps=EPS)
        out = [_held(s["k"]), _held(s["v"])]
        out += [s["k_scale"], s["v_scale"]] if s["cache"] == "e4m3" else []
        return out if q is None else out + [q]
    if s["op"] == "read":
        return list(B.cache_read(s["handle"], s["table"], s["offsets"], s["rows"], out_dtype=DT[s["y"]]))
    return B.paged_attention(s["q"], s["handle"], s["table"], s["lens"], window=s["window"], lse=s["lse"])


# -------------------------------------------------------------------------------------- work

def work(case):
    D, kv = case["D"], case["kv"]
    held = kv * (D * SIZE[case.get("cache", "bf16")] + (4 * -(-D // BLOCK) if case.get("cache") == "e4m3" else 0))
    if case["op"] == "rope":
        n = case["M"] * (case["heads"] + kv) * D
        return {"bytes": n * (SIZE[case["x"]] + SIZE[case["y"]]) + 4 * case["M"] * case["axes"], "flops": n * (6 + 4 * case["norm"])}
    if case["op"] == "write":
        M, heads, x = case["M"], case["heads"], SIZE[case["x"]]
        b = M * (2 * kv * D * x + 2 * held + 2 * heads * D * x + 8 + 4 * (case["R"] > 0))
        return {"bytes": b, "flops": M * (2 * kv + heads) * D * 8}
    tokens = sum(min(n, case.get("window") or n) for n in _lengths(case))
    if case["op"] == "read":
        return {"bytes": tokens * (2 * held + 2 * kv * D * SIZE[case["y"]]), "flops": 2 * tokens * kv * D}
    rows = case["B"] * case["heads"]
    b = 2 * tokens * held + 2 * rows * D * SIZE[case["q"]] + 4 * rows * case["lse"] + 4 * -(-tokens // case["page"])
    return {"bytes": b, "flops": 4 * tokens * case["heads"] * D}


# ------------------------------------------------------------------------------------- exact

def _nearest_e4m3(v):
    """E4M3 values of float64 values: nearest, ties to even, saturating at 448."""
    a = v.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))).clamp(min=-6.0) - 3.0)
    return torch.copysign((torch.round(a / step) * step).clamp(max=448.0), v)


def _exact_turn(x, s, weight):
    """The rotation as a product of complex numbers."""
    z = x.to(torch.float64)
    M, H, D = z.shape
    if weight is not None:
        rms = (z.square().sum(-1) / D + EPS).sqrt()
        z = z * weight.to(torch.float64) / rms[..., None]
    R = s["R"]
    if R == 0:
        return z
    half = R // 2
    first = torch.arange(half, device=z.device) * (1 if s["pairing"] == "half" else 2)
    second = first + (half if s["pairing"] == "half" else 1)
    pos = s["positions"].reshape(-1, M).to(torch.float64)
    axis = s.get("axis") or [0] * half
    angle = torch.empty(M, half, dtype=torch.float64, device=z.device)
    for i in range(half):
        angle[:, i] = pos[axis[i]] * float(s["inv_freq"][i].item())
    turned = torch.complex(z[..., first], z[..., second]) * torch.polar(torch.ones_like(angle), angle)[:, None, :]
    y = z.clone()
    y[..., first], y[..., second] = turned.real, turned.imag
    return y


def _exact_codes(y):
    """(values of the codes, scales): both are defined on the float32 values."""
    D = y.shape[-1]
    q = torch.empty_like(y)
    groups = []
    for g in range(0, D, BLOCK):
        part = y[..., g:g + BLOCK].float()
        top = part.abs().max(-1, keepdim=True).values.clamp(min=1e-10)
        scale = top / torch.full_like(top, 448.0)
        q[..., g:g + BLOCK] = _nearest_e4m3((part / scale).to(torch.float64))
        groups.append(top.to(torch.float64) / 448)
    return q, torch.cat(groups, -1)


def _exact_write(s):
    out = {n: _held(s[n]).to(torch.float64) for n in ("k", "v")}
    if s["cache"] == "e4m3":
        out.update({n: s[n].to(torch.float64) for n in ("k_scale", "v_scale")})
    slots = s["slots"].tolist()
    kept = [m for m in range(s["M"]) if slots[m] >= 0]
    page = torch.tensor([slots[m] // s["page"] for m in kept], device="cuda", dtype=torch.long)
    row = torch.tensor([slots[m] % s["page"] for m in kept], device="cuda", dtype=torch.long)
    pick = torch.tensor(kept, device="cuda", dtype=torch.long)
    for name, y in (("k", _exact_turn(s["kx"], s, s["k_weight"])), ("v", s["vx"].to(torch.float64))):
        y = y[pick]
        if s["cache"] == "e4m3":
            out[name].index_put_((page, row), _exact_codes(y)[0])
            out[name + "_scale"].index_put_((page, row), _exact_codes(y)[1])
        else:
            out[name].index_put_((page, row), y)
    res = [out["k"], out["v"]] + ([out["k_scale"], out["v_scale"]] if s["cache"] == "e4m3" else [])
    return res if s["q"] is None else res + [_exact_turn(s["q"], s, s["q_weight"])]


def _exact_rows(s, which, b, pos):
    """Float64 rows [positions, heads, D] of a sequence, one position at a time by its page and row."""
    page, row = s["table"][b].long()[pos // s["page"]], pos % s["page"]
    y = _held(s[which])[page, row].to(torch.float64)
    if s["cache"] == "e4m3":
        sc = s[which + "_scale"][page, row].to(torch.float64)
        for g in range(sc.shape[-1]):
            y[..., g * BLOCK:(g + 1) * BLOCK] *= sc[..., g:g + 1]
    return y


def _exact_read(s):
    y = [[], []]
    for b, n in enumerate(s["n"]):
        pos = torch.arange(n, device="cuda")
        for i, which in enumerate(("k", "v")):
            y[i].append(_exact_rows(s, which, b, pos))
    return [torch.cat(y[0]), torch.cat(y[1])]


def _exact_attention(s):
    B, H, kv, D = len(s["n"]), s["heads"], s["kv"], s["D"]
    G = H // kv
    y = torch.zeros(B, H, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["n"]):
        pos = torch.arange(_span(s, n), n, device="cuda")
        if n == 0:
            continue
        k, v = _exact_rows(s, "k", b, pos), _exact_rows(s, "v", b, pos)
        for h in range(kv):
            rows = slice(h * G, (h + 1) * G)
            logits = k[:, h].contiguous().matmul(s["q"][b, rows].to(torch.float64).t().contiguous()) / math.sqrt(D)
            lse[b, rows] = torch.logsumexp(logits, 0)
            y[b, rows] = torch.exp(logits - lse[b, rows]).t().contiguous().matmul(v[:, h].contiguous())
    return [y, lse] if s["lse"] else y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        y = [_exact_turn(s["q"], s, s["q_weight"])]
        return y + ([_exact_turn(s["k"], s, s["k_weight"])] if s["k"] is not None else [])
    return {"write": _exact_write, "read": _exact_read, "attention": _exact_attention}[case["op"]](s)
