"""Refusals of the rotary positions and the paged cache, before any launch (no GPU needed)."""
import ctypes

import pytest

import block_scaled_fp8_linear_amd as B

FAKE = 1 << 40
name = B.status_name


def make_cache(**kw):
    """Head-major E4M3 pages of 16 rows, 4 heads of 208 channels; ``kw`` replaces fields."""
    c = B.Cache(B.DT_F8_E4M3, 4, 208, 16, 10, FAKE, FAKE, 4 * 16 * 208, 208, 16 * 208, FAKE, FAKE, 4 * 2 * 16, 1, 32, 16)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _validate(**kw):
    return name(B.lib().bsf8_cache_validate(ctypes.byref(make_cache(**kw))))


def test_cache_descriptor():
    assert name(B.lib().bsf8_cache_validate(None)) == "INVALID_ARG"
    assert _validate() == "OK"
    assert _validate(page=16 * 4 * 208, row=4 * 208, head=208) == "OK"                       # token-major
    assert _validate(page=2 * 16 * 4 * 208, row=4 * 208, head=208) == "OK"                   # keys and values side by side
    assert _validate(dtype=B.DT_BF16, k_scale=None, v_scale=None) == "OK"
    assert _validate(n_pages=1, page=0) == "OK" and _validate(heads=1, head=0, s_head=0) == "OK"
    for bad in (dict(dtype=B.DT_F32), dict(dtype=B.DT_F8_E5M2), dict(heads=0), dict(head_dim=0), dict(page_size=0),
                dict(n_pages=0), dict(heads=-1), dict(n_pages=-5), dict(k=None), dict(v=None), dict(k_scale=None),
                dict(v_scale=None), dict(dtype=B.DT_BF16), dict(dtype=B.DT_BF16, k_scale=None), dict(page=-16), dict(row=-208),
                dict(row=176), dict(head=208), dict(page=4 * 16 * 208 - 16), dict(page=0), dict(s_row=-1), dict(s_row=0),
                dict(s_group=15), dict(s_head=16), dict(s_page=127), dict(page=1 << 62), dict(n_pages=1, page=1 << 62)):
        assert _validate(**bad) == "INVALID_ARG", bad
    for bad in (dict(k=FAKE + 8), dict(v=FAKE + 1), dict(row=216, head=16 * 216, page=64 * 216), dict(k_scale=FAKE + 2),
                dict(v_scale=FAKE + 1), dict(dtype=B.DT_BF16, k_scale=None, v_scale=None, head=16 * 208 + 4, page=1 << 14)):
        assert _validate(**bad) == "ALIGNMENT", bad
    for bad in (dict(head_dim=72), dict(head_dim=272), dict(head_dim=8), dict(n_pages=1 << 27), dict(n_pages=1 << 40),
                dict(heads=1, head=0, row=1 << 28, page=1 << 33), dict(page=1 << 32), dict(s_page=1 << 32),
                dict(s_row=1 << 26, s_head=16, s_group=64, s_page=1 << 30)):
        assert _validate(**bad) == "UNSUPPORTED", bad


def _rope(**kw):
    a = B.RopeArgs()
    a.M, a.head_dim, a.rotary_dim, a.n_axes, a.positions, a.position_bytes = 5, 64, 32, 1, FAKE, 4
    a.inv_freq, a.scale, a.eps, a.weight_dtype = FAKE, 1.0, 1e-6, B.DT_F32
    a.q = a.q_out = B.Heads(FAKE, B.DT_BF16, 3, 192, 64)
    for k, v in kw.items():
        setattr(a, k, v)
    return name(B.lib().bsf8_rope(ctypes.byref(a), None))


def H(data=FAKE, dtype=B.DT_BF16, heads=3, token=192, head=64):
    return B.Heads(data, dtype, heads, token, head)


def test_rope_refusals():
    assert name(B.lib().bsf8_rope(None, None)) == "INVALID_ARG"
    assert _rope(M=0) == "OK" and _rope(M=0, positions=None) == "OK"
    for bad in (dict(M=-1), dict(head_dim=0), dict(rotary_dim=66), dict(rotary_dim=-2), dict(rotary_dim=31), dict(pairing=2),
                dict(n_axes=0), dict(n_axes=17), dict(positions=None), dict(position_bytes=2), dict(inv_freq=None),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(axis=bytes([0] * 15 + [1])), dict(n_axes=3, axis=bytes([3] * 16)),
                dict(q=H(None)), dict(q_out=H(None)), dict(q=H(None), q_out=H(None)), dict(q=H(heads=0)),
                dict(q_out=H(heads=2)), dict(q=H(dtype=B.DT_F16)), dict(q_out=H(dtype=B.DT_U8)), dict(q=H(token=-1)),
                dict(q=H(head=-64)), dict(q_out=H(token=100)), dict(q_out=H(head=63)), dict(q_out=H(token=0)),
                dict(k=H()), dict(k_out=H()), dict(k_weight=FAKE), dict(q_weight=FAKE, eps=0.0),
                dict(q_weight=FAKE, eps=float("nan")), dict(q_weight=FAKE, weight_dtype=B.DT_F16), dict(ld_axis=-1),
                dict(q=H(token=1 << 61)), dict(q=H(None), q_out=H(None), k=H(), k_out=H(), q_weight=FAKE)):
        assert _rope(**bad) == "INVALID_ARG", bad
    for bad in (dict(q=H(FAKE + 1)), dict(q_out=H(FAKE + 1)), dict(q=H(FAKE + 2, B.DT_F32)), dict(positions=FAKE + 2),
                dict(positions=FAKE + 4, position_bytes=8), dict(inv_freq=FAKE + 2), dict(q_weight=FAKE + 2),
                dict(k=H(), k_out=H(FAKE + 1))):
        assert _rope(**bad) == "ALIGNMENT", bad
    for bad in (dict(head_dim=72), dict(head_dim=272), dict(M=1 << 31), dict(M=1 << 30)):
        assert _rope(**bad) == "UNSUPPORTED", bad


def _write(cache=None, M=5, k=H(token=832, head=208, heads=4), v=H(token=832, head=208, heads=4), slots=FAKE, b=8, rope=None):
    c = make_cache() if cache is None else cache
    ref = lambda x: ctypes.byref(x) if x is not None else None
    return name(B.lib().bsf8_cache_write(ref(c), M, ref(k), ref(v), slots, b, ref(rope), None))


def test_cache_write_refusals():
    def rope(**kw):
        a = B.RopeArgs()
        a.M, a.head_dim, a.rotary_dim, a.n_axes, a.positions, a.position_bytes = 5, 208, 64, 1, FAKE, 4
        a.inv_freq, a.scale, a.eps, a.weight_dtype = FAKE, 1.0, 1e-6, B.DT_F32
        for key, val in kw.items():
            setattr(a, key, val)
        return a

    heads = dict(token=832, head=208, heads=4)
    assert _write(M=0) == "OK" and _write(M=0, k=None, v=None, slots=None) == "OK"
    assert name(B.lib().bsf8_cache_write(None, 0, None, None, None, 8, None, None)) == "INVALID_ARG"
    for bad in (dict(cache=make_cache(heads=0)), dict(M=-1), dict(k=None), dict(v=None), dict(slots=None), dict(b=2),
                dict(k=H(token=832, head=208, heads=3)), dict(v=H(token=832, head=208, heads=5)), dict(k=H(None, **heads)),
                dict(k=H(dtype=B.DT_U8, **heads)), dict(rope=rope(M=4)), dict(rope=rope(head_dim=64)),
                dict(rope=rope(k=H(**heads))), dict(rope=rope(k_out=H(**heads))), dict(rope=rope(q=H(**heads))),
                dict(rope=rope(q_weight=FAKE)), dict(rope=rope(k_weight=FAKE, eps=-1.0)), dict(rope=rope(rotary_dim=210))):
        assert _write(**bad) == "INVALID_ARG", bad
    for bad in (dict(k=H(FAKE + 1, **heads)), dict(v=H(FAKE + 2, B.DT_F32, **heads)), dict(slots=FAKE + 4), dict(slots=FAKE + 2, b=4),
                dict(rope=rope(k_weight=FAKE + 1))):
        assert _write(**bad) == "ALIGNMENT", bad
    assert _write(M=1 << 29) == "UNSUPPORTED" and _write(M=1 << 40) == "UNSUPPORTED"
    assert _write(cache=make_cache(head_dim=72)) == "UNSUPPORTED"


def _read(cache=None, B_=3, table=FAKE, ld=8, pages=8, starts=None, off=FAKE, R=20, k=H(token=832, head=208, heads=4),
          v=H(token=832, head=208, heads=4)):
    c = make_cache() if cache is None else cache
    ref = lambda x: ctypes.byref(x) if x is not None else None
    return name(B.lib().bsf8_cache_read(ref(c), B_, table, ld, pages, starts, off, R, ref(k), ref(v), None))


def test_cache_read_refusals():
    heads = dict(token=832, head=208, heads=4)
    assert _read(B_=0) == "OK" and _read(R=0) == "OK"
    assert name(B.lib().bsf8_cache_read(None, 0, None, 0, 0, None, None, 0, None, None, None)) == "INVALID_ARG"
    for bad in (dict(B_=-1), dict(R=-1), dict(table=None), dict(ld=7), dict(pages=0), dict(pages=-1), dict(off=None),
                dict(k=None, v=None), dict(k=H(None, **heads), v=None), dict(k=H(dtype=B.DT_F32, **heads)),
                dict(v=H(token=832, head=208, heads=3)), dict(k=H(token=700, head=208, heads=4)), dict(k=H(token=0, head=208, heads=4)),
                dict(ld=1 << 61), dict(k=H(dtype=B.DT_U8, **heads))):
        assert _read(**bad) == "INVALID_ARG", bad
    for bad in (dict(table=FAKE + 2), dict(off=FAKE + 1), dict(starts=FAKE + 2), dict(k=H(FAKE + 1, **heads))):
        assert _read(**bad) == "ALIGNMENT", bad
    for bad in (dict(B_=1 << 31), dict(pages=1 << 27, ld=1 << 27), dict(R=1 << 30)):
        assert _read(**bad) == "UNSUPPORTED", bad


def test_rope_axes():
    assert B.rope_axes([2, 3, 1]) == bytes([0, 0, 1, 1, 1, 2])
    assert B.rope_axes([24, 20, 20], interleaved=True)[:7] == bytes([0, 1, 2, 0, 1, 2, 0])
    a = B.rope_axes([24, 20, 20], interleaved=True)
    assert [a.count(i) for i in range(3)] == [24, 20, 20] and a[60:] == bytes(4)
    assert B.rope_axes([5]) == bytes(5)
    for bad in ([], [1] * 17, [3, -1]):
        with pytest.raises(ValueError):
            B.rope_axes(bad)
    with pytest.raises(ValueError):
        B.rope_axes([0, 4], interleaved=True)


def _attention(cache=None, ws=FAKE, wsb=1 << 40, **kw):
    a = B.AttentionArgs()
    a.B, a.table, a.ld_table, a.pages, a.lens, a.scale = 3, FAKE, 100, 100, FAKE, 0.1
    a.q = a.out = B.Heads(FAKE, B.DT_BF16, 8, 8 * 208, 208)
    for key, val in kw.items():
        setattr(a, key, val)
    c = make_cache() if cache is None else cache
    return name(B.lib().bsf8_paged_attention(ctypes.byref(c), ctypes.byref(a), ws, wsb, None))


def test_attention_refusals():
    L = B.lib()
    wide = dict(token=8 * 208, head=208, heads=8)
    assert _attention(B=0) == "OK" and _attention(B=0, lens=None, table=None) == "OK"
    assert name(L.bsf8_paged_attention(ctypes.byref(make_cache()), None, None, 0, None)) == "INVALID_ARG"
    assert name(L.bsf8_paged_attention(None, ctypes.byref(B.AttentionArgs()), None, 0, None)) == "INVALID_ARG"
    for bad in (dict(cache=make_cache(heads=0)), dict(B=-1), dict(window=-1), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(q=H(heads=6, token=8 * 208, head=208)), dict(q=H(heads=0, token=8 * 208, head=208)), dict(q=H(None, **wide)),
                dict(out=H(heads=4, token=8 * 208, head=208)), dict(out=H(None, **wide)), dict(q=H(dtype=B.DT_F16, **wide)),
                dict(out=H(dtype=B.DT_F8_E4M3, **wide)), dict(out=H(heads=8, token=8 * 208 - 1, head=208)), dict(table=None),
                dict(lens=None), dict(pages=0), dict(ld_table=99)):
        assert _attention(**bad) == "INVALID_ARG", bad
    for bad in (dict(table=FAKE + 2), dict(lens=FAKE + 1), dict(lse=FAKE + 2), dict(q=H(FAKE + 1, **wide)), dict(out=H(FAKE + 1, **wide)),
                dict(ws=FAKE + 128)):
        assert _attention(**bad) == "ALIGNMENT", bad
    for bad in (dict(B=1 << 31), dict(B=1 << 22, ld_table=1 << 30), dict(pages=1 << 27, ld_table=1 << 27), dict(B=1 << 20, pages=1 << 20, ld_table=1 << 20)):
        assert _attention(**bad) == "UNSUPPORTED", bad
    need = ctypes.c_size_t()
    assert L.bsf8_attention_workspace_size(ctypes.byref(make_cache()), 3, 8, 100, ctypes.byref(need)) == 0 and need.value > 0
    assert _attention(ws=None) == "WORKSPACE" and _attention(wsb=need.value - 1) == "WORKSPACE"
    for bad in (dict(q=6), dict(q=0), dict(B=-1), dict(pages=0)):
        kw = dict(dict(B=3, q=8, pages=100), **bad)
        assert name(L.bsf8_attention_workspace_size(ctypes.byref(make_cache()), kw["B"], kw["q"], kw["pages"], ctypes.byref(need))) == "INVALID_ARG"
        assert need.value == 0
    assert name(L.bsf8_attention_workspace_size(ctypes.byref(make_cache()), 3, 8, 100, None)) == "INVALID_ARG"
    assert L.bsf8_attention_workspace_size(ctypes.byref(make_cache()), 3, 8, 2, ctypes.byref(need)) == 0 and need.value == 0
    assert L.bsf8_attention_workspace_size(ctypes.byref(make_cache()), 0, 8, 100, ctypes.byref(need)) == 0 and need.value == 0


def test_workspace_covers_every_type_of_query():
    """The workspace is asked for without the query's type; whatever it is, a call that joins finds room (the call checks
    the same number)."""
    L, need = B.lib(), ctypes.c_size_t()
    for D in (64, 128, 144, 256):
        for b in (1, 3, 40, 700):
            for pages in (1, 9, 33, 70, 400, 5000):
                c = make_cache(head_dim=D, row=D, head=16 * D, page=64 * D)
                assert L.bsf8_attention_workspace_size(ctypes.byref(c), b, 8, pages, ctypes.byref(need)) == 0
                assert need.value <= 64 << 20


@pytest.mark.parametrize("current,owner", [(0, 1), (1, 0), (1, 1)])
def test_workspace_is_asked_on_the_caches_device(monkeypatch, current, owner):
    import types

    import torch
    state, seen = [current], []

    class Guard:
        def __init__(self, idx):
            self.idx = idx

        def __enter__(self):
            self.old, state[0] = state[0], self.idx

        def __exit__(self, *exc):
            state[0] = self.old

    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(B, "_CURRENT", (lambda: state[0], lambda idx: 0))
    monkeypatch.setattr(B, "lib", lambda: types.SimpleNamespace(bsf8_attention_workspace_size=lambda *a: seen.append(state[0]) or 0))
    cache = types.SimpleNamespace(_idx=owner, _ref=None)
    assert B.attention_workspace_size(cache, 3, 8, 100) == 0
    assert seen == [owner] and state == [current]


def test_copied_axes_are_read_where_the_copy_keeps_them():
    """What the library reads of a copied or pickled RopeAxes is the copy's own memory, which outlives the original's."""
    import copy
    import pickle

    axes = B.rope_axes([2, 3, 1])
    held = {"axes": axes}
    for other in (copy.copy(axes), copy.deepcopy(axes), copy.deepcopy(held)["axes"], pickle.loads(pickle.dumps(axes)),
                  pickle.loads(pickle.dumps(axes, 0))):
        assert type(other) is B.RopeAxes and other == axes
        assert other.address == ctypes.addressof(other._held) and bytes(other._held) == bytes(other)
    assert copy.deepcopy(axes).address != axes.address


def test_no_tokens_with_head_weights():
    """An empty tensor has no address, so without tokens a weight is not refused for want of its heads: rope, and a cache's
    queries and keys."""
    none = H(None)
    for kw in (dict(q_weight=FAKE), dict(k_weight=FAKE), dict(q_weight=FAKE, k_weight=FAKE), dict(q_out=H(), q_weight=FAKE),
               dict(k_out=H(), k_weight=FAKE)):
        kw = dict(dict(q_out=none), **kw)
        assert _rope(M=0, q=none, **kw) == "OK", kw
        assert _rope(M=5, q=none, **kw) == "INVALID_ARG", kw
    for kw in (dict(q_weight=FAKE), dict(q_weight=FAKE, k_weight=FAKE), dict(q_out=H(heads=4), q_weight=FAKE)):
        for M, want in ((0, "OK"), (5, "INVALID_ARG")):
            a = B.RopeArgs()
            a.M, a.head_dim, a.rotary_dim, a.n_axes, a.positions, a.position_bytes = M, 208, 64, 1, FAKE, 4
            a.inv_freq, a.scale, a.eps, a.weight_dtype = FAKE, 1.0, 1e-6, B.DT_F32
            for key, val in kw.items():
                setattr(a, key, val)
            assert _write(M=M, rope=a) == want, kw
    # what is wrong whatever the tokens stays refused
    assert _rope(M=0, q=none, q_out=none, q_weight=FAKE, eps=0.0) == "INVALID_ARG"
    assert _rope(M=0, q=none, q_out=none, k_weight=FAKE, weight_dtype=B.DT_F16) == "INVALID_ARG"


def test_the_binding_without_tokens_and_with_head_weights(monkeypatch):
    """The same through the binding, which passes an empty tensor's address (host tensors, nothing is launched)."""
    import types

    import torch
    monkeypatch.setattr(B, "_CURRENT", (lambda: -1, lambda idx: 0))
    monkeypatch.setattr(B, "_gpu_index", lambda name, t: -1)
    monkeypatch.setattr(B, "_T", torch)
    x = torch.randn(3, 12, 208)
    q, k, v = x[:0, :4], x[:0, 4:8], x[:0, 8:]
    assert q.data_ptr() == 0
    w, inv, pos = torch.ones(208), torch.ones(32), torch.arange(3)[:0]
    for kw in (dict(q_weight=w), dict(k=k, k_weight=w), dict(k=k, q_weight=w, k_weight=w, k_out=torch.empty(0, 4, 208))):
        y, yk = B.rope(q, pos, inv, **kw)
        assert y.shape == (0, 4, 208) and (yk is None) == ("k" not in kw)
    c = make_cache()
    cache = types.SimpleNamespace(_idx=-1, heads=4, head_dim=208, _ref=ctypes.byref(c))
    y = B.cache_write(cache, k, v, pos, positions=pos, inv_freq=inv, q=q, q_weight=w, k_weight=w)
    assert y.shape == (0, 4, 208)
    assert B.cache_write(cache, k, v, pos, positions=pos, inv_freq=inv, k_weight=w) is None
