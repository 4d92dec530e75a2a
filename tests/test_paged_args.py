"""Refusals of the rotary positions and the paged cache, on the host: the
binding's checks of types and shapes and the C ABI's checks before any device
work."""
import ctypes
import math

import pytest
import torch

import log_domain_sinkhorn_amd as sk

BF, I32 = torch.bfloat16, torch.int32


def test_frequencies():
    f = sk.rotary_frequencies(64, device="cpu")
    assert f.dtype == torch.float64 and f.shape == (32,)
    i = torch.arange(32, dtype=torch.float64)
    assert torch.allclose(f, 10000.0 ** (-2 * i / 64), rtol=1e-14)
    assert torch.allclose(sk.rotary_frequencies(64, factor=4.0, device="cpu"), f / 4, rtol=1e-14)
    g = sk.rotary_frequencies(64, factor=4.0, original_length=8192, low=1.0, high=32.0, device="cpu")
    turns = 8192 * f / (2 * math.pi)
    assert torch.allclose(g[turns >= 32], f[turns >= 32], rtol=1e-14) and (turns >= 32).any()
    assert torch.allclose(g[turns <= 1], f[turns <= 1] / 4, rtol=1e-14) and (turns <= 1).any()
    mid = (turns > 1) & (turns < 32)
    keep = (turns[mid] - 1) / 31
    assert torch.allclose(g[mid], f[mid] * (keep + (1 - keep) / 4), rtol=1e-13) and mid.any()
    assert sk.rotary_frequencies(0, device="cpu").shape == (0,)
    for bad in (dict(rotated=3), dict(rotated=-2), dict(base=0.0), dict(base=math.nan), dict(factor=0.0),
                dict(factor=math.inf), dict(original_length=-1.0), dict(original_length=8.0, low=2.0, high=2.0),
                dict(original_length=8.0, low=math.nan)):
        kw = {"rotated": 64, **bad}
        with pytest.raises(sk.SinkhornError):
            sk.rotary_frequencies(kw.pop("rotated"), device="cpu", **kw)
    assert sk.lib().sinkhorn_rotary_frequencies(4, 1e4, 1.0, 0.0, 1.0, 32.0, None) == sk.ERR_INVALID_ARG


def _rot(**kw):
    a = dict(q=torch.zeros(2, 3, 4, 8, dtype=BF), k=torch.zeros(2, 3, 2, 8, dtype=BF),
             frequencies=torch.ones(4, dtype=torch.float64))
    a.update(kw)
    return a


@pytest.mark.parametrize("bad", [
    dict(q=torch.zeros(2, 3, 4, 8, dtype=torch.float64)), dict(k=torch.zeros(2, 3, 2, 8)), dict(q=None), dict(q=[1.0]),
    dict(frequencies=torch.ones(4)), dict(positions=torch.zeros(2, 3)), dict(positions=torch.zeros(2, 3, dtype=torch.int64)),
    dict(norm_eps=1e-6, q_weight=torch.ones(8, dtype=torch.float16)), dict(norm_eps=1e-6, q_weight=torch.ones(8, dtype=torch.float64)),
    dict(norm_eps=1e-6, q_weight=torch.ones(8), k_weight=torch.ones(8, dtype=BF)), dict(lengths=torch.zeros(2)),
    dict(q_out=torch.zeros(2, 3, 4, 8)),
])
def test_rotation_types(bad):
    with pytest.raises(TypeError):
        sk.rotate_heads(**_rot(**bad))


@pytest.mark.parametrize("bad", [
    dict(q=torch.zeros(3, 4, 8, dtype=BF)), dict(k=torch.zeros(2, 4, 2, 8, dtype=BF)), dict(k=torch.zeros(2, 3, 2, 16, dtype=BF)),
    dict(frequencies=torch.ones(5, dtype=torch.float64)), dict(frequencies=torch.ones(1, 4, dtype=torch.float64)),
    dict(frequencies=torch.ones(8, dtype=torch.float64)[::2]), dict(positions=torch.zeros(3, 2, dtype=I32)),
    dict(positions=torch.zeros(2, dtype=I32)), dict(positions=torch.zeros(3, 2, dtype=I32).t()),
    dict(frequencies=None, positions=torch.zeros(3, dtype=I32)), dict(q_weight=torch.ones(8)),
    dict(norm_eps=1e-6, q_weight=torch.ones(4)), dict(k=None, norm_eps=1e-6, k_weight=torch.ones(8)),
    dict(lengths=torch.zeros(3, dtype=I32)), dict(q_out=torch.zeros(2, 3, 4, 4, dtype=BF)),
    dict(q_out=torch.zeros(1, 3, 4, 8, dtype=BF).expand(2, 3, 4, 8)), dict(k=None, k_out=torch.zeros(2, 3, 2, 8, dtype=BF)),
    dict(q=torch.zeros(2, 3, 4, 8, dtype=BF, requires_grad=True)), dict(frequencies=torch.ones(4, dtype=torch.float64, requires_grad=True)),
    dict(norm_eps=1e-6, q_weight=torch.ones(8, requires_grad=True)), dict(q=torch.zeros(2, 3, 8, 4, dtype=BF).transpose(2, 3)),
    dict(),  # host tensors
])
def test_rotation_shapes_and_places(bad):
    with pytest.raises(ValueError):
        sk.rotate_heads(**_rot(**bad))


def test_rotation_gradient_arguments():
    a = _rot()
    q, k, f = a["q"], a["k"], a["frequencies"]
    for kw in (dict(norm_eps=1e-6), dict(norm_eps=1e-6, q=q), dict(norm_eps=1e-6, q=q, k=q), dict(norm_eps=1e-6, q=q[:, :2], k=k),
               dict(dq=k), dict()):
        with pytest.raises(ValueError):
            sk.rotate_heads_grad(q, k, frequencies=f, **kw)
    with pytest.raises(TypeError):
        sk.rotate_heads_grad(q, k, q.float(), k, frequencies=f, norm_eps=1e-6)


def _app(**kw):
    a = dict(k=torch.zeros(2, 3, 2, 8, dtype=BF), v=torch.zeros(2, 3, 2, 16, dtype=BF), k_cache=torch.zeros(4, 8, 2, 8, dtype=BF),
             v_cache=torch.zeros(4, 8, 2, 16, dtype=BF), page_table=torch.zeros(2, 2, dtype=I32),
             cache_lengths=torch.zeros(2, dtype=I32))
    a.update(kw)
    return a


@pytest.mark.parametrize("bad", [
    dict(v=torch.zeros(2, 3, 2, 16)), dict(k_cache=torch.zeros(4, 8, 2, 8)), dict(page_table=torch.zeros(2, 2, dtype=torch.int64)),
    dict(page_table=None), dict(cache_lengths=torch.zeros(2, dtype=torch.int64)), dict(new_lengths=torch.zeros(2)),
    dict(q=torch.zeros(2, 3, 4, 8)), dict(lengths_out=torch.zeros(2)),
])
def test_append_types(bad):
    with pytest.raises(TypeError):
        sk.cache_append(**_app(**bad))


@pytest.mark.parametrize("bad", [
    dict(v=torch.zeros(2, 2, 2, 16, dtype=BF)), dict(v=torch.zeros(2, 3, 2, 8, dtype=BF)), dict(k_cache=torch.zeros(4, 8, 1, 8, dtype=BF)),
    dict(k_cache=torch.zeros(4, 8, 2, 16, dtype=BF)), dict(v_cache=torch.zeros(4, 4, 2, 16, dtype=BF)),
    dict(v_cache=torch.zeros(5, 8, 2, 16, dtype=BF)), dict(page_table=torch.zeros(3, 2, dtype=I32)),
    dict(page_table=torch.zeros(2, dtype=I32)), dict(page_table=torch.zeros(2, 2, dtype=I32).t()),
    dict(cache_lengths=torch.zeros(3, dtype=I32)), dict(new_lengths=torch.zeros(1, dtype=I32)), dict(q=torch.zeros(2, 4, 4, 8, dtype=BF)),
    dict(q_weight=torch.ones(8), norm_eps=1e-6), dict(q_out=torch.zeros(2, 3, 2, 8, dtype=BF)),
    dict(k_cache=torch.zeros(1, 8, 2, 8, dtype=BF).expand(4, 8, 2, 8)), dict(lengths_out=torch.zeros(3, dtype=I32)), dict(),
])
def test_append_shapes_and_places(bad):
    with pytest.raises(ValueError):
        sk.cache_append(**_app(**bad))


AT = [ctypes.c_void_p(1 << 40 | i << 34) for i in range(24)]  # addresses far apart, never read


def _desc(**kw):
    r = sk._RotationC(dtype=2, batch=2, heads_q=4, heads_kv=2, d=64, rotated=64, len=3, gain=1.0, eps=1e-6, frequencies=AT[20].value,
                      weight_dtype=0)
    for n in ("q", "k", "q_out", "k_out", "dq", "dk"):
        setattr(r, n + "_stride", sk._i64x3(4096, 512, 64))
    for n, x in kw.items():
        setattr(r, n, x)
    return r


def _rotate(r, q=AT[0], k=AT[1], qw=None, kw=None, qo=AT[2], ko=AT[3]):
    return sk.lib().sinkhorn_rotate_heads(ctypes.byref(r) if r else None, q, k, qw, kw, qo, ko, None)


def _grad(r, dqo=AT[0], dko=AT[1], q=AT[2], k=AT[3], qw=None, kw=None, dq=AT[4], dk=AT[5], wq=AT[6], wk=AT[7], ws=AT[8], n=1 << 30):
    return sk.lib().sinkhorn_rotate_heads_grad(ctypes.byref(r) if r else None, dqo, dko, q, k, qw, kw, dq, dk, wq, wk, ws, n, None)


@pytest.mark.parametrize("kw,word", [
    (dict(dtype=3), b"dtype"), (dict(batch=-1), b"negative"), (dict(len=-1), b"negative"), (dict(heads_q=0, heads_kv=0), b"heads"),
    (dict(heads_q=-1), b"heads"), (dict(d=0), b"width"), (dict(rotated=65), b"rotated"), (dict(rotated=3), b"rotated"), (dict(rotated=-2), b"rotated"),
    (dict(gain=math.nan), b"gain"), (dict(gain=1e39), b"gain"), (dict(norm=1, eps=-1.0), b"eps"), (dict(norm=1, eps=math.inf), b"eps"),
    (dict(weight_dtype=1), b"weights"), (dict(len=1 << 30), b"2^31"), (dict(frequencies=None), b"frequencies"),
    (dict(q_stride=sk._i64x3(-1, 1, 1)), b"stride"), (dict(position_stride=-1), b"stride"),
])
def test_rotation_descriptions_are_refused(kw, word):
    r = _desc(**kw)
    n = ctypes.c_int64()
    assert _rotate(r) == sk.ERR_INVALID_ARG and word in sk.lib().sinkhorn_last_error()
    assert _grad(r) == sk.ERR_INVALID_ARG and word in sk.lib().sinkhorn_last_error()
    assert sk.lib().sinkhorn_rotation_workspace(ctypes.byref(r), ctypes.byref(n)) == sk.ERR_INVALID_ARG


def test_rotation_pointers_overlaps_and_workspaces():
    L = sk.lib()
    assert _rotate(None) == sk.ERR_INVALID_ARG and _grad(None) == sk.ERR_INVALID_ARG
    assert _rotate(_desc(d=129)) == sk.ERR_UNSUPPORTED and _rotate(_desc(heads_q=8193)) == sk.ERR_UNSUPPORTED
    for kw in (dict(q=None), dict(k=None), dict(qo=None), dict(ko=None)):
        assert _rotate(_desc(), **kw) == sk.ERR_INVALID_ARG, kw
    near = lambda p, n=128: ctypes.c_void_p(p.value + n)  # noqa: E731
    # an output that is another argument, or lies across it; in place only with the same strides
    for kw in (dict(qo=AT[1]), dict(ko=AT[2]), dict(qo=near(AT[0])), dict(qo=AT[20]), dict(qw=AT[2]), dict(kw=AT[3])):
        assert _rotate(_desc(), **kw) == sk.ERR_INVALID_ARG, kw
        assert b"overlaps" in L.sinkhorn_last_error()
    assert _rotate(_desc(q_out_stride=sk._i64x3(8192, 512, 64)), qo=AT[0]) == sk.ERR_INVALID_ARG
    assert _rotate(_desc(positions=AT[2].value)) == sk.ERR_INVALID_ARG
    assert _rotate(_desc(lengths=AT[3].value)) == sk.ERR_INVALID_ARG
    r = _desc(norm=1)
    n = ctypes.c_int64()
    assert L.sinkhorn_rotation_workspace(ctypes.byref(r), ctypes.byref(n)) == sk.OK and n.value > 0
    assert L.sinkhorn_rotation_workspace(ctypes.byref(r), None) == sk.ERR_INVALID_ARG
    for kw in (dict(dqo=None), dict(dko=None), dict(q=None), dict(k=None), dict(dq=None), dict(dk=None), dict(ws=None),
               dict(n=n.value - 1), dict(ws=near(AT[8], 8)), dict(dq=AT[2]), dict(dk=AT[0]), dict(wq=AT[7]), dict(wq=AT[4]), dict(ws=AT[6]),
               dict(qw=AT[6])):
        assert _grad(r, **kw) == sk.ERR_INVALID_ARG, kw
    assert _grad(_desc(norm=1, heads_kv=0), dko=None, k=None, dk=None) == sk.ERR_INVALID_ARG  # dk_weight without keys
    assert _grad(_desc()) == sk.ERR_INVALID_ARG  # gradients of weights without a norm
    # nothing to do needs no device
    assert _rotate(_desc(batch=0), None, None, None, None, None, None) == sk.OK
    assert _grad(_desc(len=0), None, None, None, None, None, None, None, None, None, None, None, 0) == sk.OK


def _pages(**kw):
    c = sk._PagesC(page_size=16, table_len=4, pages=10, table_stride=4, dv=64, page_table=AT[10].value, lengths=AT[11].value,
                   k_stride=sk._i64x3(8192, 512, 64), v_stride=sk._i64x3(8192, 512, 64))
    for n, x in kw.items():
        setattr(c, n, x)
    return c


def _append(r, c, q=AT[0], k=AT[1], v=AT[2], vs=sk._i64x3(4096, 512, 64), qw=None, kw=None, qo=AT[3], kc=AT[4], vc=AT[5], lo=AT[6]):
    return sk.lib().sinkhorn_cache_append(ctypes.byref(r) if r else None, ctypes.byref(c) if c else None, q, k, v, vs, qw, kw, qo, kc,
                                          vc, lo, None)


def test_append_refusals():
    L = sk.lib()
    assert _append(None, _pages()) == sk.ERR_INVALID_ARG and _append(_desc(), None) == sk.ERR_INVALID_ARG
    for kw, word in ((dict(page_size=0), b"page_size"), (dict(page_size=12), b"page_size"), (dict(page_size=-8), b"page_size"),
                     (dict(table_len=-1), b"negative"), (dict(pages=-1), b"negative"), (dict(table_stride=-1), b"negative"),
                     (dict(table_len=1 << 27), b"2^31"), (dict(pages=1 << 31), b"2^31"), (dict(dv=0), b"width"),
                     (dict(k_stride=sk._i64x3(1, -1, 1)), b"stride"), (dict(page_table=None), b"null"), (dict(lengths=None), b"null")):
        assert _append(_desc(), _pages(**kw)) == sk.ERR_INVALID_ARG, kw
        assert word in L.sinkhorn_last_error(), kw
    assert _append(_desc(), _pages(dv=129)) == sk.ERR_UNSUPPORTED
    assert _append(_desc(heads_kv=0), _pages()) == sk.ERR_INVALID_ARG
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(vs=None), dict(qo=None), dict(kc=None), dict(vc=None), dict(lo=None),
               dict(vs=sk._i64x3(-1, 1, 1))):
        assert _append(_desc(), _pages(), **kw) == sk.ERR_INVALID_ARG, kw
    for kw in (dict(kc=AT[5]), dict(kc=AT[1]), dict(vc=AT[2]), dict(qo=AT[1]), dict(lo=AT[11]), dict(lo=AT[10]), dict(lo=AT[4]),
               dict(kc=AT[10]), dict(qo=AT[4])):
        assert _append(_desc(), _pages(), **kw) == sk.ERR_INVALID_ARG, kw
        assert b"overlaps" in L.sinkhorn_last_error(), kw
    assert _append(_desc(batch=0), _pages()) == sk.OK


def test_append_without_a_table():
    """A cache of no pages needs a table too where a token is appended: its places are looked up there."""
    L = sk.lib()
    for kw in (dict(pages=0), dict(pages=0, table_len=1), dict()):
        assert _append(_desc(), _pages(page_table=None, **kw)) == sk.ERR_INVALID_ARG, kw
        assert b"page table" in L.sinkhorn_last_error(), kw
    assert _append(_desc(batch=0), _pages(pages=0, page_table=None)) == sk.OK


def _att(**kw):
    a = dict(q=torch.zeros(2, 3, 4, 8, dtype=BF), k_cache=torch.zeros(4, 8, 2, 8, dtype=BF), v_cache=torch.zeros(4, 8, 2, 16, dtype=BF),
             page_table=torch.zeros(2, 2, dtype=I32), key_lengths=torch.zeros(2, dtype=I32))
    a.update(kw)
    return a


@pytest.mark.parametrize("bad", [
    dict(q=torch.zeros(2, 3, 4, 8)), dict(q=[1]), dict(k_cache=torch.zeros(4, 8, 2, 8)), dict(v_cache=None), dict(page_table=torch.zeros(2, 2)),
    dict(key_lengths=torch.zeros(2)), dict(query_lengths=torch.zeros(2, dtype=torch.int64)), dict(out=torch.zeros(2, 3, 4, 16)),
    dict(lse=torch.zeros(2, 4, 3, dtype=torch.float64)),
])
def test_paged_attention_types(bad):
    with pytest.raises(TypeError):
        sk.paged_attention(**_att(**bad))


@pytest.mark.parametrize("bad", [
    dict(q=torch.zeros(2, 3, 8, dtype=BF)), dict(q=torch.zeros(2, 3, 3, 8, dtype=BF)), dict(q=torch.zeros(2, 3, 4, 16, dtype=BF)),
    dict(k_cache=torch.zeros(4, 8, 16, dtype=BF)), dict(k_cache=torch.zeros(4, 8, 0, 8, dtype=BF)),
    dict(v_cache=torch.zeros(4, 8, 1, 16, dtype=BF)), dict(page_table=torch.zeros(1, 2, dtype=I32)),
    dict(key_lengths=torch.zeros(1, dtype=I32)), dict(query_lengths=torch.zeros(3, dtype=I32)), dict(recent=0), dict(recent=-1),
    dict(first=2), dict(out=torch.zeros(2, 3, 4, 8, dtype=BF)), dict(out=torch.zeros(1, 3, 4, 16, dtype=BF).expand(2, 3, 4, 16)),
    dict(lse=torch.zeros(2, 3, 4)), dict(q=torch.zeros(2, 3, 4, 8, dtype=BF, requires_grad=True)),
    dict(k_cache=torch.zeros(4, 8, 2, 8, dtype=BF, requires_grad=True)), dict(),
])
def test_paged_attention_shapes_and_places(bad):
    with pytest.raises(ValueError):
        sk.paged_attention(**_att(**bad))


def _adesc(**kw):
    a = sk._AttentionC(dtype=2, batch=2, heads_q=4, heads_kv=2, d=64, dv=64, len_q=3, scale=0.125)
    for n in ("q", "out"):
        setattr(a, n + "_stride", sk._i64x3(4096, 512, 64))
    for n, x in kw.items():
        setattr(a, n, x)
    return a


def _attend(a, c, first=0, recent=0, q=AT[0], k=AT[1], v=AT[2], out=AT[3], lse=AT[4], ws=AT[5], n=1 << 30):
    return sk.lib().sinkhorn_paged_attention(ctypes.byref(a) if a else None, ctypes.byref(c) if c else None, first, recent, q, k, v, out,
                                             lse, ws, n, None)


def test_paged_attention_refusals():
    L = sk.lib()
    assert _attend(None, _pages()) == sk.ERR_INVALID_ARG and _attend(_adesc(), None) == sk.ERR_INVALID_ARG
    for kw, word in ((dict(dtype=5), b"dtype"), (dict(batch=-1), b"negative"), (dict(heads_kv=3), b"multiple"), (dict(d=0), b"width"),
                     (dict(scale=0.0), b"scale"), (dict(dv=32), b"dv"), (dict(len_q=1 << 30), b"2^31"), (dict(key_bias=AT[9].value), b"key_bias"),
                     (dict(key_lengths=AT[9].value), b"key_lengths")):
        assert _attend(_adesc(**kw), _pages()) == sk.ERR_INVALID_ARG, kw
        assert word in L.sinkhorn_last_error(), kw
    for kw in (dict(page_size=20), dict(table_len=-1), dict(page_table=None), dict(lengths=None), dict(v_stride=sk._i64x3(-1, 1, 1))):
        assert _attend(_adesc(), _pages(**kw)) == sk.ERR_INVALID_ARG, kw
    for kw in (dict(first=-1), dict(recent=-1), dict(first=3), dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(lse=None)):
        assert _attend(_adesc(), _pages(), **kw) == sk.ERR_INVALID_ARG, kw
    # rows that are not whole, aligned units of 16 bytes, and slots too far apart
    for at, c in ((_adesc(d=60), _pages()), (_adesc(dv=60), _pages(dv=60)), (_adesc(), _pages(k_stride=sk._i64x3(8192, 516, 64))),
                  (_adesc(), _pages(v_stride=sk._i64x3(8192, 512, 68))), (_adesc(d=136), _pages()), (_adesc(), _pages(v_stride=sk._i64x3(0, 1 << 27, 64)))):
        assert _attend(at, c) == sk.ERR_UNSUPPORTED
    assert _attend(_adesc(), _pages(), k=ctypes.c_void_p(AT[1].value + 8)) == sk.ERR_UNSUPPORTED
    for kw in (dict(out=AT[1]), dict(out=AT[0]), dict(lse=AT[3]), dict(lse=AT[11]), dict(out=AT[10])):
        assert _attend(_adesc(), _pages(), **kw) == sk.ERR_INVALID_ARG, kw
        assert b"overlaps" in L.sinkhorn_last_error(), kw
    # a long table is split: it takes a workspace
    c, n = _pages(table_len=4096, table_stride=4096), ctypes.c_int64()
    assert L.sinkhorn_paged_workspace(ctypes.byref(_adesc()), ctypes.byref(c), 0, 0, ctypes.byref(n)) == sk.OK and n.value > 0
    whole = n.value
    assert L.sinkhorn_paged_workspace(ctypes.byref(_adesc()), ctypes.byref(c), 4, 100, ctypes.byref(n)) == sk.OK and n.value < whole
    assert L.sinkhorn_paged_workspace(ctypes.byref(_adesc()), ctypes.byref(c), 0, 0, None) == sk.ERR_INVALID_ARG
    for kw in (dict(ws=None), dict(n=whole - 1), dict(ws=ctypes.c_void_p(AT[5].value + 8))):
        assert _attend(_adesc(), c, **kw) == sk.ERR_INVALID_ARG and b"workspace" in L.sinkhorn_last_error()
    assert _attend(_adesc(), c, ws=AT[1]) == sk.ERR_INVALID_ARG and b"overlaps" in L.sinkhorn_last_error()
    assert _attend(_adesc(batch=0), _pages()) == sk.OK
    assert _attend(_adesc(len_q=0), _pages()) == sk.OK


def test_sizes_beyond_the_descriptions():
    """Sizes that the C side's fields do not hold are the caller's error like any other."""
    many = 1 << 31
    with pytest.raises(ValueError, match="size"):  # slots of a page
        wide = torch.zeros(1, 1, 2, 8, dtype=BF).expand(1, many, 2, 8)
        sk.paged_attention(**_att(k_cache=wide, v_cache=wide))
    with pytest.raises(ValueError, match="size"):  # pages of a sequence
        sk.cache_append(**_app(page_table=torch.empty(0, many, dtype=I32), k=torch.zeros(0, 3, 2, 8, dtype=BF),
                               v=torch.zeros(0, 3, 2, 16, dtype=BF), cache_lengths=torch.zeros(0, dtype=I32)))
    # sequences (on the device: here the descriptions alone)
    for pack, n in ((sk._pack_rotation, 34), (sk._pack_attention, 38)):
        with pytest.raises(ValueError, match="size"):
            pack(0, many, *[0] * (n - 2))
