"""Rotary positions, the paged cache and its attention as programs use them: a run of them between the projections, decode
steps from a graph, several calls at once, other streams, and memory beyond 32 bits."""
import numpy as np
import pytest

import block_scaled_fp8_linear_amd as B
import synth
from cache_util import attention64, cache_values, make_table, new_cache, rope64, rope_tolerance, to_f64
from gpu_util import banner, device, member_to_device, torch

pytestmark = pytest.mark.gpu


class Block:
    """The attention half of a transformer block: norm, grouped Q/K/V, rotation and cache, attention, output projection."""
    H, KV, D, K, page = 6, 2, 128, 512, 16

    def __init__(self, seqs, pages_each, codes=True):
        t = torch()
        H, KV, D, K = self.H, self.KV, self.D, self.K
        members = [synth.random_code_weight(901, n, r, K) for n, r in (("q", H * D), ("k", KV * D), ("v", KV * D))]
        self.qkv = B.BlockFP8Weight([member_to_device(m) for m in members])
        self.o = B.BlockFP8Weight([member_to_device(synth.random_code_weight(901, "o", K, H * D))])
        self.norm = t.rand(K, device=device()) + 0.5
        self.head_norm = (1 + 0.1 * t.randn(D, device=device())).bfloat16()
        self.inv = (1e4 ** (-t.arange(0, D, 2, device=device(), dtype=t.float64) / D)).float()
        self.axes = B.rope_axes([24, 20, 20], interleaved=True)
        self.cache = B.PagedKVCache.new(seqs * pages_each + 1, self.page, KV, D, None if codes else t.bfloat16, device())
        g = np.random.default_rng(5)
        self.table = t.from_numpy(g.permutation(seqs * pages_each).reshape(seqs, pages_each).astype(np.int32)).to(device())

    def step(self, x, lens, keep=None):
        """One new token per sequence, at position lens - 1; lens, x [seqs, K] on the GPU."""
        t = torch()
        H, KV, D = self.H, self.KV, self.D
        xq, xs, h, _ = B.quant_norm(x, self.norm, residual=x, h=t.empty_like(x))
        y = B.linear_w8a8(self.qkv, xq, xs).unflatten(1, (H + 2 * KV, D))
        pos = lens - 1
        slot = self.table.gather(1, (pos // self.page).long()[:, None])[:, 0] * self.page + pos % self.page
        q, k, v = y[:, :H], y[:, H:H + KV], y[:, H + KV:]
        three = t.stack([pos, pos // 3, pos % 7]).contiguous()
        q = B.cache_write(self.cache, k, v, slot, positions=three, inv_freq=self.inv, axes=self.axes, q=q,
                          q_weight=self.head_norm, k_weight=self.head_norm)
        a = B.paged_attention(q, self.cache, self.table, lens)
        aq, as_ = B.quant_act(a.flatten(1))
        out = B.linear_w8a8_epilogue(self.o, aq, as_, residual=h, out_dtype=t.float32)
        if keep is not None:
            keep.update(y=y, q=q, three=three, slot=slot, a=a)
        return out


@pytest.mark.parametrize("codes", [True, False])
def test_a_block_step_by_step(codes):
    """Forty decode steps: each step's rotation, stored rows and attention against their definitions."""
    t = torch()
    seqs = 5
    blk = Block(seqs, 6, codes)
    g = np.random.default_rng(6)
    lens = np.array([1, 30, 50, 17, 2])
    for b, n in enumerate(lens):            # what earlier steps have left
        for p in range(n - 1):
            s = int(blk.table[b, p // 16]) * 16 + p % 16
            kv = t.randn(1, 2 * blk.KV, blk.D, device=device())
            B.cache_write(blk.cache, kv[:, :blk.KV], kv[:, blk.KV:], t.tensor([s], device=device()))
    for step in range(40):
        x = t.from_numpy(g.standard_normal((seqs, blk.K)).astype(np.float32)).to(device())
        keep = {}
        if step % 10 == 0:
            banner(f"block step {step} codes={codes}")
        out = blk.step(x, t.from_numpy(lens.astype(np.int32)).to(device()), keep)
        assert out.shape == (seqs, blk.K) and bool(t.isfinite(out).all())
        if step % 13 == 0:
            y, w = to_f64(keep["y"]), to_f64(blk.head_norm)
            want = rope64(y[:, :blk.H], keep["three"].cpu().numpy(), blk.inv.cpu().numpy(), blk.axes, weight=w)
            assert (np.abs(to_f64(keep["q"]) - want) <= rope_tolerance(want, y[:, :blk.H], weight=w, bf16=True)).all()
            vals = cache_values(blk.cache)
            slot = keep["slot"].cpu().numpy()
            k = rope64(y[:, blk.H:blk.H + blk.KV], keep["three"].cpu().numpy(), blk.inv.cpu().numpy(), blk.axes, weight=w)
            for got, ref in ((vals[0], k), (vals[1], y[:, blk.H + blk.KV:])):
                got = got[slot // 16, slot % 16]
                top = np.abs(ref).max(-1, keepdims=True)
                step_of = 2.0 ** -4 * np.abs(ref) + top / 448 * 2.0 ** -10 if codes else 2.0 ** -8 * np.abs(ref)
                assert (np.abs(got - ref) <= step_of + 2.0 ** -20 * top).all()
            want, _, tol, _ = attention64(to_f64(keep["q"]), vals, blk.table.cpu().numpy(), lens, 16, 0, blk.D ** -0.5,
                                          blk.cache.n_pages)
            assert (np.abs(to_f64(keep["a"]) - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol)).all()
        lens = lens + 1


def test_decode_steps_from_a_graph():
    """A captured step follows new tokens, lengths and slots: every replay equals the eager step on a cache of its own, with
    eager work between the replays."""
    t = torch()
    seqs = 4
    a, b = Block(seqs, 70), Block(seqs, 70)
    assert t.equal(a.table, b.table)
    b.norm, b.head_norm = a.norm, a.head_norm
    g = np.random.default_rng(7)
    lens = np.array([1, 300, 1000, 40])
    for blk in (a, b):
        t.manual_seed(3)
        codes = t.randint(0, 120, blk.cache.k.transpose(1, 2).shape, dtype=t.uint8, device=device())
        for x in (blk.cache.k, blk.cache.v):
            x.copy_(codes.transpose(1, 2))
        for s in (blk.cache.k_scale, blk.cache.v_scale):
            s.fill_(0.004)
    x = t.zeros(seqs, a.K, device=device())
    ln = t.ones(seqs, dtype=t.int32, device=device())
    assert B.attention_workspace_size(a.cache, seqs, a.H, 70) > 0
    warm = Block(seqs, 70)
    warm.step(x, ln)
    t.cuda.synchronize()
    banner("graph of a decode step")
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        y = a.step(x, ln)
    a.cache.k.copy_(b.cache.k), a.cache.v.copy_(b.cache.v)
    a.cache.k_scale.copy_(b.cache.k_scale), a.cache.v_scale.copy_(b.cache.v_scale)
    for step in range(12):
        x.copy_(t.from_numpy(g.standard_normal((seqs, a.K)).astype(np.float32)))
        ln.copy_(t.from_numpy(lens.astype(np.int32)))
        graph.replay()
        got = y.clone()
        want = b.step(x, ln)
        t.cuda.synchronize()
        assert t.equal(got, want), step
        assert t.equal(a.cache.k, b.cache.k) and t.equal(a.cache.v_scale, b.cache.v_scale)
        lens = lens + np.array([1, 1, 7, 60])


def _attention_case(seed, lens, codes=True, D=128, H=16, KV=4):
    t = torch()
    g = np.random.default_rng(seed)
    pages = sum(-(-n // 16) for n in lens) + 1
    cache, _ = new_cache("head_major", pages, 16, KV, D, codes)
    if codes:
        cache.k_scale.mul_(0.01), cache.v_scale.mul_(0.01)
    table = t.from_numpy(make_table(g, lens, 16, pages)).to(device())
    q = t.from_numpy(g.standard_normal((len(lens), H, D)).astype(np.float32)).to(device()).bfloat16()
    return q, cache, table, t.tensor(lens, dtype=t.int32, device=device())


def test_two_graphs_of_one_stream_at_once():
    """Both join parts and were captured on one stream; replayed together on two streams, each with its own workspace."""
    t = torch()
    cases = [_attention_case(1, [5000, 3, 900]), _attention_case(2, [700, 4000])]
    graphs, outs, wants = [], [], []
    banner("two attention graphs")
    for c in cases:
        assert B.attention_workspace_size(c[1], c[0].shape[0], 16, c[2].shape[1]) > 0
        out = t.empty_like(c[0])
        B.paged_attention(*c, out=out)
        wants.append(out.clone())
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph):
            B.paged_attention(*c, out=out)
        graphs.append(graph)
        outs.append(out)
    streams = [t.cuda.Stream(), t.cuda.Stream()]
    for _ in range(4):
        for out in outs:
            out.zero_()
        t.cuda.synchronize()
        for _ in range(5):
            for graph, st in zip(graphs, streams):
                with t.cuda.stream(st):
                    graph.replay()
        t.cuda.synchronize()
        assert all(t.equal(o, w) for o, w in zip(outs, wants))


def test_calls_on_two_streams_at_once():
    t = torch()
    cases = [_attention_case(3, [4000, 17]), _attention_case(4, [90, 2500, 1], codes=False)]
    x = [t.randn(200, 12, 128, device=device()) for _ in range(2)]
    inv = t.rand(64, device=device())
    pos = t.arange(200, device=device())
    slots = t.randperm(13 * 16, device=device())[:200]

    def go(i):
        c = cases[i]
        cache = B.PagedKVCache.new(13, 16, 2, 128, device=device())
        q = B.cache_write(cache, x[i][:, 8:10], x[i][:, 10:], slots, positions=pos, inv_freq=inv, q=x[i][:, :8])
        k, v = B.cache_read(cache, t.arange(13, dtype=t.int32, device=device())[None], t.tensor([0, 200], dtype=t.int32, device=device()), 200)
        return [B.paged_attention(*c), q, k, v, cache.k_scale] + [y for y in B.rope(x[i], pos, inv) if y is not None]

    banner("attention on two streams")
    wants = [go(i) for i in range(2)]
    t.cuda.synchronize()
    streams = [t.cuda.Stream(), t.cuda.Stream()]
    for _ in range(5):
        got = []
        for i, st in enumerate(streams):
            with t.cuda.stream(st):
                got.append(go(i))
        t.cuda.synchronize()
        for a, b in zip(got, wants):
            assert all(t.equal(p, q) for p, q in zip(a, b))


def test_given_workspace():
    t = torch()
    q, cache, table, lens = _attention_case(5, [3000, 40])
    want = B.paged_attention(q, cache, table, lens)
    need = B.attention_workspace_size(cache, 2, 16, table.shape[1])
    ws = t.full((need,), 0xFF, dtype=t.uint8, device=device())     # NaN wherever it is read as floats
    guard = t.full((need + 512,), 0x5A, dtype=t.uint8, device=device())
    for w in (ws, guard[256:256 + need]):
        for _ in range(2):
            assert t.equal(B.paged_attention(q, cache, table, lens, workspace=(w, need)), want)
    assert bool((guard[:256] == 0x5A).all()) and bool((guard[256 + need:] == 0x5A).all())
    with pytest.raises(ValueError):
        B.paged_attention(q, cache, table, lens, workspace=(ws, need + 1))
    with pytest.raises(B.BSF8Error, match="WORKSPACE"):
        B.paged_attention(q, cache, table, lens, workspace=(ws, need - 1))
    with pytest.raises(B.BSF8Error, match="WORKSPACE"):
        B.paged_attention(q, cache, table, lens, workspace=(None, 0))


@pytest.mark.parametrize("codes", [True, False])
def test_cache_beyond_32_bits(codes):
    """Pages whose bytes lie beyond 2^32, and pages almost 2^32 bytes apart."""
    t = torch()
    dt = t.uint8 if codes else t.bfloat16
    D, KV, page = 128, 2, 16
    size = 1 if codes else 2
    n_pages = (6 << 30) // (page * KV * D * size)
    for far in (False, True):
        if far:
            n_pages, step = 4, (((1 << 32) - 4096) // size) // 16 * 16
            base = t.zeros(3 * step + page * KV * D, dtype=dt, device=device())
            kv = [base.as_strided((n_pages, page, KV, D), (step, D, page * D, 1))] * 2
        else:
            kv = [t.zeros(n_pages, KV, page, D, dtype=dt, device=device()).transpose(1, 2) for _ in "kv"]
        sc = [t.ones(n_pages, KV, 1, page, device=device()).permute(0, 3, 1, 2) for _ in "kv"] if codes else []
        cache = B.PagedKVCache(*kv, *sc)
        pages = [n_pages - 1, 1, n_pages - 2, 0]
        table = t.tensor([pages], dtype=t.int32, device=device())
        n = 55
        pos = t.arange(n, device=device())
        slots = table[0].long()[pos // page] * page + pos % page
        x = t.randn(n, 2 * KV, D, device=device()).bfloat16()
        banner(f"cache beyond 32 bits codes={codes} far={far}")
        # (one tensor for both where pages lie far apart: the values are written last, and are the keys too)
        B.cache_write(cache, x[:, KV:] if far else x[:, :KV], x[:, KV:], slots)
        k, v = B.cache_read(cache, table, t.tensor([0, n], dtype=t.int32, device=device()), n, out_dtype=t.float32)
        small = B.PagedKVCache.new(4, page, KV, D, dtype=dt, device=device())
        near = t.arange(4, dtype=t.int32, device=device())[None]
        B.cache_write(small, x[:, KV:] if far else x[:, :KV], x[:, KV:], pos)
        wk, wv = B.cache_read(small, near, t.tensor([0, n], dtype=t.int32, device=device()), n, out_dtype=t.float32)
        assert t.equal(k, wk) and t.equal(v, wv)
        q = t.randn(1, 8, D, device=device()).bfloat16()
        ln = t.tensor([n], dtype=t.int32, device=device())
        assert t.equal(B.paged_attention(q, cache, table, ln), B.paged_attention(q, small, near, ln))
        del cache, kv, sc
        t.cuda.empty_cache()


def test_many_sequences():
    """More sequences than a wave counts at a time, with every few empty; items by block and by item."""
    t = torch()
    g = np.random.default_rng(9)
    lens = [int(n) if i % 5 else 0 for i, n in enumerate(g.integers(1, 40, 3000))]
    lens[2999] = 9000
    pages = sum(-(-n // 16) for n in lens) + 1
    cache, _ = new_cache("head_major", pages, 16, 1, 64, True)
    cache.k_scale.mul_(0.01), cache.v_scale.mul_(0.01)
    table = make_table(g, lens, 16, pages)
    q = t.randn(3000, 2, 64, device=device()).bfloat16()
    banner("paged_attention of 3000 sequences")
    out = B.paged_attention(q, cache, t.from_numpy(table).to(device()), t.tensor(lens, dtype=t.int32, device=device()))
    want, _, tol, _ = attention64(to_f64(q), cache_values(cache), table, lens, 16, 0, 0.125, pages)
    assert (np.abs(to_f64(out) - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol)).all()


def test_mixed_types_and_many_tokens():
    """Queries and keys of different types in one call; more tokens than fill the device several times over."""
    t = torch()
    g = np.random.default_rng(10)
    inv = (1e4 ** (-np.arange(0, 64, 2) / 64)).astype(np.float32)
    f = t.from_numpy(inv).to(device())
    q, k = t.randn(70, 5, 64, device=device()).bfloat16(), t.randn(70, 3, 64, device=device())
    p = t.arange(70, device=device())
    yq, yk = B.rope(q, p, f, k=k)
    assert yq.dtype == t.bfloat16 and yk.dtype == t.float32
    assert t.equal(yq, B.rope(q, p, f)[0]) and t.equal(yk, B.rope(k, p, f)[0])
    M = 70000
    x0 = t.randn(97, 3, 64, device=device()).bfloat16()
    idx = t.arange(M, device=device()) % 97
    banner("rope of 70000 tokens")
    want, _ = B.rope(x0, t.arange(97, device=device()), f)
    got, _ = B.rope(x0[idx], idx, f)
    assert t.equal(got, want[idx])
    cache = B.PagedKVCache.new(M // 16 + 1, 16, 3, 64, device=device())
    B.cache_write(cache, x0[idx], x0[idx], t.arange(M, device=device()), positions=idx, inv_freq=f)
    tab = t.arange(M // 16 + 1, dtype=t.int32, device=device())[None]
    k, v = B.cache_read(cache, tab, t.tensor([0, M], dtype=t.int32, device=device()), M)
    assert t.equal(k, k[:97][idx]) and t.equal(v, v[:97][idx])


def test_more_tokens_than_one_launch():
    """Tokens that repeat: every repetition of the first ones gives their bits."""
    t = torch()
    M, n = (1 << 25) + 70, 991
    x0 = t.randn(n, 1, 16, device=device()).bfloat16()
    f = t.rand(8, device=device())
    idx = t.arange(M, device=device()) % n
    banner(f"rope of {M} tokens")
    want, _ = B.rope(x0, t.arange(n, device=device()), f)
    x = x0[idx]
    got, _ = B.rope(x, idx, f, out=x)
    assert t.equal(got, want[idx])


def test_refusals_of_the_binding():
    t = torch()
    d = device()
    q, cache, table, lens = _attention_case(6, [30, 20])
    x = t.randn(2, 4, 128, device=d)
    pos, inv = t.arange(2, device=d), t.ones(64, device=d)
    slots = t.arange(2, device=d)
    off = t.tensor([0, 4, 9], dtype=t.int32, device=d)
    bad = [
        lambda: B.PagedKVCache(cache.k, cache.v), lambda: B.PagedKVCache(cache.k, cache.v, cache.k_scale),
        lambda: B.PagedKVCache(cache.k, cache.v[:, :8], cache.k_scale, cache.v_scale),
        lambda: B.PagedKVCache(cache.k, cache.v, cache.k_scale, cache.v_scale.contiguous()),
        lambda: B.PagedKVCache(cache.k.float(), cache.v.float()) if False else B.PagedKVCache(cache.k.half(), cache.v.half(), cache.k_scale, cache.v_scale),
        lambda: B.PagedKVCache(cache.k.cpu(), cache.v.cpu(), cache.k_scale, cache.v_scale),
        lambda: B.rope(x[0], pos, inv), lambda: B.rope(x.half(), pos, inv), lambda: B.rope(x, pos.float(), inv),
        lambda: B.rope(x, pos[:1], inv), lambda: B.rope(x, pos, inv.double()), lambda: B.rope(x, pos, None),
        lambda: B.rope(x, None, inv), lambda: B.rope(x, pos, inv, axes=bytes(63)), lambda: B.rope(x, t.stack([pos, pos]), inv),
        lambda: B.rope(x, pos, inv, pairing="other"), lambda: B.rope(x, pos, inv, k_weight=inv), lambda: B.rope(x, pos, inv, q_weight=inv),
        lambda: B.rope(x, pos, inv, out_dtype=t.float16), lambda: B.rope(x, pos, inv, out=x[:1]), lambda: B.rope(x, pos.cpu(), inv),
        lambda: B.rope(x.transpose(1, 2), pos, inv), lambda: B.rope(x, pos, inv, out=x, out_dtype=t.bfloat16),
        lambda: B.cache_write(cache, x, x, slots.float()), lambda: B.cache_write(cache, x, x[:1], slots),
        lambda: B.cache_write(cache, x[:, :3], x[:, :3], slots), lambda: B.cache_write(cache, x, x, slots, out=x),
        lambda: B.cache_write(cache, x, x, slots, axes=bytes(64)), lambda: B.cache_write(cache, x, x, slots, q_weight=inv),
        lambda: B.cache_write(cache, x, x.cpu(), slots), lambda: B.cache_write(cache, x, x, slots, q=x[:, :, :64], positions=pos, inv_freq=inv),
        lambda: B.cache_read(cache, table.long(), off, 9), lambda: B.cache_read(cache, table, off.long(), 9),
        lambda: B.cache_read(cache, table[:1], off, 9), lambda: B.cache_read(cache, table, off, -1),
        lambda: B.cache_read(cache, table, off, 9, out_dtype=t.float16), lambda: B.cache_read(cache, table, off, 9, k_out=x),
        lambda: B.paged_attention(q[0], cache, table, lens), lambda: B.paged_attention(q[:, :, :64], cache, table, lens),
        lambda: B.paged_attention(q[:, :6], cache, table, lens), lambda: B.paged_attention(q.half(), cache, table, lens),
        lambda: B.paged_attention(q, cache, table.long(), lens), lambda: B.paged_attention(q, cache, table, lens.long()),
        lambda: B.paged_attention(q, cache, table[:1], lens), lambda: B.paged_attention(q, cache, table, lens[:1]),
        lambda: B.paged_attention(q, cache, table, lens.cpu()), lambda: B.paged_attention(q, cache, table, lens, out=x),
        lambda: B.paged_attention(q, cache, table, lens, out_dtype=t.float16),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, B.BSF8Error)):
            call()
            raise AssertionError(f"call {i} went through")
    for call in (lambda: B.paged_attention(q, cache, table, lens, window=-1), lambda: B.paged_attention(q, cache, table, lens, scale=float("nan")),
                 lambda: B.rope(x, t.stack([pos, pos]), inv, axes=bytes([0] * 63 + [2]))):
        with pytest.raises(B.BSF8Error, match="INVALID_ARG"):
            call()


@pytest.mark.parametrize("D", [64, 128, 144, 256])
@pytest.mark.parametrize("codes", [True, False])
def test_the_workspace_holds_every_type_of_query(D, codes):
    """The bytes that are asked for without the query's type are enough for each: calls that join write nothing behind them."""
    t = torch()
    joined = 0
    for lens, heads, kv in (([3000], 4, 1), ([9000, 5, 700], 8, 2), ([600] * 40, 4, 4), ([1500, 2000] * 12, 20, 1)):
        q, cache, table, ln = _attention_case(D, lens, codes, D, heads, kv)
        need = B.attention_workspace_size(cache, len(lens), heads, table.shape[1])
        joined += need > 0
        guard = t.full((need + 512 + (1 << 20),), 0x5A, dtype=t.uint8, device=device())
        ws = guard[256:256 + need]
        for dt in (t.bfloat16, t.float32):
            for out_dt in (t.bfloat16, t.float32):
                banner(f"workspace of {need} bytes D={D} codes={codes} {lens[:3]} x {len(lens)} {dt} -> {out_dt}")
                want = B.paged_attention(q.to(dt), cache, table, ln, out_dtype=out_dt)
                got = B.paged_attention(q.to(dt), cache, table, ln, out_dtype=out_dt, workspace=(ws if need else None, need))
                assert t.equal(got, want)
                assert bool((guard[:256] == 0x5A).all()) and bool((guard[256 + need:] == 0x5A).all())
    assert joined >= 2


def test_types_that_are_no_cache():
    """Caches of other types are refused, with scales and without."""
    t = torch()
    sc = [t.ones(3, 16, 2, 1, device=device()) for _ in "kv"]
    for dt in (t.float32, t.float16, t.int8, t.float8_e5m2):
        kv = [t.zeros(3, 16, 2, 64, device=device()).to(dt) for _ in "kv"]
        for scales in ([], sc, sc[:1]):
            with pytest.raises((ValueError, B.BSF8Error)):
                B.PagedKVCache(*kv, *scales)
    bf = [t.zeros(3, 16, 2, 64, device=device(), dtype=t.bfloat16) for _ in "kv"]
    u8 = [t.zeros(3, 16, 2, 64, device=device(), dtype=t.uint8) for _ in "kv"]
    for args in (bf + sc, bf + sc[:1], u8, u8 + sc[:1], [bf[0], u8[0]], [u8[0], bf[0]] + sc, u8 + [sc[0], sc[1].double()],
                 u8 + [sc[0], sc[1][:2]]):
        with pytest.raises((ValueError, B.BSF8Error)):
            B.PagedKVCache(*args)
    B.PagedKVCache(*bf), B.PagedKVCache(*u8, *sc)


def test_no_tokens_with_head_norms():
    """A step without tokens of a model with head norms does nothing."""
    t = torch()
    cache, held = new_cache("head_major", 2, 4, 2, 64, True)
    before = [h.clone() for h in held]
    x = t.randn(3, 8, 64, device=device()).bfloat16()
    w, inv = t.ones(64, device=device()), t.ones(32, device=device())
    pos, q, k, v = t.arange(3, device=device())[:0], x[:0, :4], x[:0, 4:6], x[:0, 6:]
    y, yk = B.rope(q, pos, inv, k=k, q_weight=w, k_weight=w)
    assert y.shape == (0, 4, 64) and yk.shape == (0, 2, 64)
    assert B.rope(q, pos, inv, q_weight=w)[0].shape == (0, 4, 64)
    y = B.cache_write(cache, k, v, pos, positions=pos, inv_freq=inv, q=q, q_weight=w, k_weight=w)
    assert y.shape == (0, 4, 64) and y.dtype == t.bfloat16
    t.cuda.synchronize()
    for a, b in zip(before, held):
        assert t.equal(a.view(t.uint8), b.view(t.uint8))
