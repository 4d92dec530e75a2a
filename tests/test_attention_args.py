"""Refusals of the attention operators, on the host: the binding's checks of
types and shapes and the C ABI's checks before any device work."""
import ctypes
import math

import pytest
import torch

import log_domain_sinkhorn_amd as sk

BF = torch.bfloat16


def _qkv(B=2, Lq=3, Hq=4, Hkv=2, Lk=5, d=8, dv=8, dtype=BF):
    return (torch.zeros(B, Lq, Hq, d, dtype=dtype), torch.zeros(B, Lk, Hkv, d, dtype=dtype),
            torch.zeros(B, Lk, Hkv, dv, dtype=dtype))


@pytest.mark.parametrize("change", [
    lambda a: a.update(q=a["q"].double()),
    lambda a: a.update(k=a["k"].float()),
    lambda a: a.update(q=[1.0]),
    lambda a: a.update(key_bias=torch.zeros(2, 5, dtype=BF)),
    lambda a: a.update(key_lengths=torch.ones(2, dtype=torch.int64)),
    lambda a: a.update(mass_out=torch.zeros(2, 2, 5, dtype=torch.float64)),
])
def test_wrong_types(change):
    q, k, v = _qkv()
    a = dict(q=q, k=k, v=v)
    change(a)
    with pytest.raises(TypeError):
        sk.cross_attention(**a)


@pytest.mark.parametrize("change", [
    lambda a: a.update(q=a["q"][0]),
    lambda a: a.update(k=a["k"][:1]),
    lambda a: a.update(k=a["k"][..., :4]),
    lambda a: a.update(v=a["v"][:, :4]),
    lambda a: a.update(v=a["v"][:, :, :1]),
    lambda a: a.update(q=a["q"][:, :, :3]),
    lambda a: a.update(q=a["q"].transpose(2, 3).contiguous().transpose(2, 3)),
    lambda a: a.update(key_bias=torch.zeros(2, 6)),
    lambda a: a.update(key_bias=torch.zeros(2, 1, 5)),
    lambda a: a.update(key_bias=torch.zeros(5, 2).t()),
    lambda a: a.update(key_lengths=torch.ones(3, dtype=torch.int32)),
    lambda a: a.update(query_lengths=torch.ones(2, 1, dtype=torch.int32)),
    lambda a: a.update(out=torch.zeros(2, 3, 4, 9, dtype=BF)),
    lambda a: a.update(out=torch.zeros(1, 3, 4, 8, dtype=BF).expand(2, 3, 4, 8)),
    lambda a: a.update(lse=torch.zeros(2, 3, 4)),
    lambda a: a.update(mass_in=torch.zeros(2, 2, 5)),
    lambda a: a.update(row_weight=torch.zeros(2, 3)),
    lambda a: a.update(mass_out=torch.zeros(2, 4, 5)),
    lambda a: a.update(q=a["q"].requires_grad_()),
    lambda a: a.update(key_bias=torch.zeros(2, 5, requires_grad=True)),
    lambda a: a,  # host tensors
])
def test_wrong_shapes_and_places(change):
    q, k, v = _qkv()
    a = dict(q=q, k=k, v=v)
    change(a)
    with pytest.raises(ValueError):
        sk.cross_attention(**a)


def test_gradient_and_weight_arguments():
    q, k, v = _qkv()
    out, lse = torch.zeros(2, 3, 4, 8, dtype=BF), torch.zeros(2, 4, 3)
    for bad in (dict(dout=out.float()), dict(lse=lse.double())):
        with pytest.raises(TypeError):
            sk.cross_attention_grad(**{**dict(dout=out, q=q, k=k, v=v, out=out, lse=lse), **bad})
    for bad in (dict(dout=out[:, :2]), dict(out=out[..., :4]), dict(lse=lse[:, :2]), dict(dk=q), dict()):
        with pytest.raises(ValueError):
            sk.cross_attention_grad(**{**dict(dout=out, q=q, k=k, v=v, out=out, lse=lse), **bad})
    with pytest.raises(ValueError):
        sk.attention_mass(q, k, lse[:, :1])


@pytest.mark.parametrize("bad", [dict(keep=0), dict(mass=torch.zeros(2, 2, 4)), dict(v=torch.zeros(2, 4, 2, 8, dtype=BF)),
                                 dict(k_out=torch.zeros(2, 4, 2, 8, dtype=BF)),
                                 dict(index_out=torch.zeros(2, 2, 4, dtype=torch.int32)), dict()])
def test_evict_arguments(bad):
    _, k, v = _qkv()
    with pytest.raises(ValueError):
        sk.cache_evict(**{**dict(k=k, v=v, mass=torch.zeros(2, 2, 5), keep=3), **bad})


def _desc(**kw):
    a = sk._AttentionC(dtype=2, batch=2, heads_q=4, heads_kv=2, d=64, dv=64, len_q=3, len_k=1000, scale=0.125)
    for n in ("q", "k", "v", "out", "dout", "dq", "dk", "dv"):
        setattr(a, n + "_stride", sk._i64x3(1 << 20, 256, 64))
    for n, x in kw.items():
        setattr(a, n, x)
    return a


FAKE = ctypes.c_void_p(256)


def _forward(a, q=FAKE, k=FAKE, v=FAKE, out=ctypes.c_void_p(512), lse=FAKE, w=None, mi=None, mo=None, ws=None, n=0):
    return sk.lib().sinkhorn_cross_attention(ctypes.byref(a) if a is not None else None, q, k, v, out, lse, w, mi, mo, ws,
                                             n, None)


@pytest.mark.parametrize("kw,word", [
    (dict(dtype=3), b"dtype"), (dict(batch=-1), b"negative"), (dict(len_k=-1), b"negative"), (dict(heads_kv=3), b"multiple"),
    (dict(heads_kv=0), b"multiple"), (dict(d=0), b"width"), (dict(len_k=1 << 31), b"2^31"), (dict(len_q=1 << 30), b"2^31"),
    (dict(scale=0.0), b"scale"), (dict(scale=-1.0), b"scale"), (dict(scale=math.nan), b"scale"),
    (dict(scale=math.inf), b"scale"), (dict(scale=1e-60), b"scale"), (dict(scale=1e39), b"scale"),
    (dict(k_stride=sk._i64x3(1, -64, 1)), b"stride"),
])
def test_descriptions_are_refused(kw, word):
    n = ctypes.c_int64()
    a = _desc(**kw)
    assert _forward(a) == sk.ERR_INVALID_ARG
    assert word in sk.lib().sinkhorn_last_error()
    assert sk.lib().sinkhorn_attention_workspace(ctypes.byref(a), 0, None, None, None, None, ctypes.byref(n)) == sk.ERR_INVALID_ARG


def test_wide_heads_are_unsupported():
    assert _forward(_desc(d=129)) == sk.ERR_UNSUPPORTED
    assert _forward(_desc(dv=256)) == sk.ERR_UNSUPPORTED
    assert _forward(_desc(heads_q=16384, heads_kv=8192)) == sk.ERR_UNSUPPORTED


def test_null_pointers_aliases_and_workspaces():
    L = sk.lib()
    a = _desc(len_k=1 << 16)
    assert _forward(None) == sk.ERR_INVALID_ARG
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(lse=None), dict(out=FAKE), dict(mi=FAKE),
               dict(w=FAKE)):
        assert _forward(a, **kw) == sk.ERR_INVALID_ARG, kw
    need = ctypes.c_int64()
    for what in range(4):
        assert L.sinkhorn_attention_workspace(ctypes.byref(a), what, None, None, None, None, ctypes.byref(need)) == sk.OK
    assert L.sinkhorn_attention_workspace(ctypes.byref(a), 4, None, None, None, None, ctypes.byref(need)) == sk.ERR_INVALID_ARG
    assert L.sinkhorn_attention_workspace(ctypes.byref(a), 0, None, None, None, None, None) == sk.ERR_INVALID_ARG
    assert L.sinkhorn_attention_workspace(ctypes.byref(a), 0, FAKE, FAKE, FAKE, None, ctypes.byref(need)) == sk.OK
    assert need.value > 0  # few rows against many keys: split
    odd = ctypes.c_int64()
    assert L.sinkhorn_attention_workspace(ctypes.byref(a), 0, FAKE, ctypes.c_void_p(258), FAKE, None, ctypes.byref(odd)) == sk.OK
    assert odd.value == need.value + 2 * 2 * (1 << 16) * 2 * 64  # a copy of k
    for ws, n in ((None, 0), (FAKE, need.value - 1), (ctypes.c_void_p(264), need.value)):
        assert _forward(a, ws=ws, n=n) == sk.ERR_INVALID_ARG
        assert b"workspace" in L.sinkhorn_last_error()
    P = [FAKE] * 3
    out, dout, dq, dk, dv = (ctypes.c_void_p(512 * i) for i in range(2, 7))
    grad = lambda *x: L.sinkhorn_cross_attention_grad(ctypes.byref(a), *x, None, 0, None)  # noqa: E731
    assert grad(*P, out, FAKE, dout, None, dk, dv) == sk.ERR_INVALID_ARG
    assert grad(*P, out, FAKE, dout, dq, dq, dv) == sk.ERR_INVALID_ARG
    assert grad(*P, out, FAKE, dout, dq, dk, dout) == sk.ERR_INVALID_ARG
    assert grad(*P, out, FAKE, dout, dq, dk, dv) == sk.ERR_INVALID_ARG  # no workspace
    assert b"workspace" in L.sinkhorn_last_error()
    assert L.sinkhorn_attention_mass(ctypes.byref(a), FAKE, FAKE, FAKE, None, None, None, None, 0, None) == sk.ERR_INVALID_ARG
    # nothing to do needs no device
    a0 = _desc(batch=0)
    assert _forward(a0) == sk.OK


def _cache(**kw):
    c = sk._CacheC(dtype=1, batch=1, heads=2, d=64, dv=64, len=100, keep=10, first=1, recent=2)
    for n in ("k", "v", "k_out", "v_out"):
        setattr(c, n + "_stride", sk._i64x3(12800, 128, 64))
    for n, x in kw.items():
        setattr(c, n, x)
    return c


def test_cache_descriptions_are_refused():
    L = sk.lib()
    p = [ctypes.c_void_p(4096 * i) for i in range(1, 9)]
    call = lambda c, *x, ws=p[7], n=1 << 20: L.sinkhorn_cache_evict(  # noqa: E731
        ctypes.byref(c) if c else None, *x, ws, n, None)
    assert call(None, *p) == sk.ERR_INVALID_ARG
    for kw in (dict(dtype=7), dict(batch=-1), dict(heads=0), dict(len=-1), dict(len=1 << 31), dict(keep=0), dict(first=-1),
               dict(recent=-1), dict(first=9, recent=2), dict(first=1 << 62, recent=1 << 62), dict(d=0),
               dict(v_out_stride=sk._i64x3(1, -1, 1))):
        assert call(_cache(**kw), *p) == sk.ERR_INVALID_ARG, kw
    for i in range(8):
        q = list(p)
        q[i] = None
        assert call(_cache(), *q) == sk.ERR_INVALID_ARG, i
    for i, j in ((3, 0), (4, 1), (4, 3), (5, 2)):
        q = list(p)
        q[i] = q[j]
        assert call(_cache(), *q) == sk.ERR_INVALID_ARG, (i, j)
    need = ctypes.c_int64()
    assert L.sinkhorn_cache_workspace(ctypes.byref(_cache()), ctypes.byref(need)) == sk.OK and need.value > 0
    assert L.sinkhorn_cache_workspace(ctypes.byref(_cache(keep=0)), ctypes.byref(need)) == sk.ERR_INVALID_ARG
    assert L.sinkhorn_cache_workspace(ctypes.byref(_cache()), None) == sk.ERR_INVALID_ARG
    for kw in (dict(ws=None), dict(n=need.value - 1), dict(ws=ctypes.c_void_p(4104))):
        assert call(_cache(), *p, **kw) == sk.ERR_INVALID_ARG and b"workspace" in L.sinkhorn_last_error()
    assert call(_cache(batch=0), *([None] * 8)) == sk.OK


def test_overlapping_side_outputs_are_refused():
    """Arrays that some workgroups read while others write."""
    L = sk.lib()
    at = lambda x: ctypes.c_void_p(x)  # noqa: E731
    a = _desc()  # weights of 2 * 2 * 1000 floats, lse of 2 * 4 * 3, row weights of 2 * 3
    for kw in (dict(mi=at(1 << 20), mo=at((1 << 20) + 16000 - 4)), dict(mi=at((1 << 20) + 4), mo=at(1 << 20)),
               dict(mo=at(1 << 20), lse=at((1 << 20) + 15996)), dict(mo=at(1 << 20), lse=at((1 << 20) - 92)),
               dict(mo=at(1 << 20), w=at((1 << 20) + 96)), dict(mo=at(1 << 20), mi=at(1 << 21), lse=at((1 << 21) + 32)),
               dict(mo=at(1 << 20), w=at(1 << 21), lse=at((1 << 21) + 20))):
        assert _forward(a, **kw) == sk.ERR_INVALID_ARG and b"overlaps" in L.sinkhorn_last_error(), kw
    for kw in (dict(mi=at(1 << 20), mo=at(1 << 20)), dict(mi=at(1 << 20), mo=at((1 << 20) + 16000)),
               dict(mo=at(1 << 20), lse=at((1 << 20) - 96), w=at((1 << 20) + 16000))):
        assert _forward(a, **kw) == sk.ERR_INVALID_ARG and b"workspace" in L.sinkhorn_last_error(), kw
    own = lambda lse, w, mi, mo: L.sinkhorn_attention_mass(ctypes.byref(a), FAKE, FAKE, lse, w, mi, mo, None, 0, None)  # noqa: E731
    assert own(at(1 << 20), None, None, at(1 << 20)) == sk.ERR_INVALID_ARG and b"overlaps" in L.sinkhorn_last_error()
    assert own(FAKE, None, at((1 << 20) + 64), at(1 << 20)) == sk.ERR_INVALID_ARG and b"overlaps" in L.sinkhorn_last_error()
    # k, v, mass, k_out, v_out, mass_out, index_out, lengths_out
    p = [at(1 << (20 + i)) for i in range(8)]
    lens = at(1 << 30)
    evict = lambda c, *x: L.sinkhorn_cache_evict(ctypes.byref(c), *x, None, 0, None)  # noqa: E731
    for i, x in ((7, 1 << 30), (5, (1 << 22) + 796), (6, 1 << 22), (7, (1 << 22) + 8), (6, (1 << 25) + 76), (7, 1 << 25),
                 (7, (1 << 26) + 40), (5, (1 << 30) - 76), (3, 1 << 21), (4, 1 << 20)):
        q = list(p)
        q[i] = at(x)
        assert evict(_cache(key_lengths=lens), *q) == sk.ERR_INVALID_ARG, (i, x)
        assert b"overlaps" in L.sinkhorn_last_error() or b"aliases" in L.sinkhorn_last_error(), (i, x)
    assert evict(_cache(key_lengths=lens), *p) == sk.ERR_INVALID_ARG and b"workspace" in L.sinkhorn_last_error()


def _fill(a):
    """Arguments of every entry point far apart from each other, and a workspace
    that suffices: {name: address}."""
    names = ("q", "k", "v", "out", "lse", "w", "mi", "mo", "dout", "dq", "dk", "dv", "bias", "qlen", "klen", "ws")
    at = {n: (i + 1) << 36 for i, n in enumerate(names)}
    a.key_bias, a.query_lengths, a.key_lengths = at["bias"], at["qlen"], at["klen"]
    a.bias_stride = sk._i64x2(1000, 0)
    return at


def _call_all(a, at, n):
    """What each entry point says: the launch itself fails where there is no device."""
    L, r, res = sk.lib(), ctypes.byref(a), {}
    p = lambda *names: [ctypes.c_void_p(at[x]) for x in names]  # noqa: E731
    for name, code in (
            ("forward", lambda: L.sinkhorn_cross_attention(r, *p("q", "k", "v", "out", "lse", "w", "mi", "mo", "ws"), n, None)),
            ("grad", lambda: L.sinkhorn_cross_attention_grad(
                r, *p("q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv", "ws"), n, None)),
            ("mass", lambda: L.sinkhorn_attention_mass(r, *p("q", "k", "lse", "w", "mi", "mo", "ws"), n, None))):
        c = code()
        res[name] = c == sk.ERR_INVALID_ARG and any(x in L.sinkhorn_last_error() for x in (b"overlap", b"alias"))
    return res


@pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that are no memory: only where nothing can be launched")
def test_arrays_that_share_memory_are_refused():
    """By elements: [2][3 or 1000][4 or 2][64] of bf16, rows 512 bytes apart."""
    n = 1 << 30
    FW, GR, MA = {"forward"}, {"grad"}, {"mass"}
    for change, want in (
            (dict(), set()),
            # a part of another array's elements
            (dict(out="q", by=128), FW), (dict(out="k", by=512 * 999 + 128), FW), (dict(out="v", by=256 - 2), FW),
            (dict(lse="q", by=512 * 2), FW), (dict(lse="k", by=4), FW), (dict(mo="q", by=0), FW | MA),
            (dict(mo="k", by=512 * 900), FW | MA), (dict(mo="bias", by=7996), FW | MA), (dict(mo="klen", by=4), FW | MA),
            (dict(mo="out", by=256), FW), (dict(lse="out", by=0), FW), (dict(lse="klen", by=4), FW),
            (dict(out="bias", by=4000), FW), (dict(mo="mi", by=0), set()),
            (dict(dq="q", by=384), GR), (dict(dk="k", by=128), GR), (dict(dv="k", by=512), GR), (dict(dk="dout", by=0), GR),
            (dict(dv="dk", by=126), GR), (dict(dq="out", by=2), GR), (dict(dk="lse", by=92), GR), (dict(dv="bias", by=0), GR),
            (dict(dq="qlen", by=0), GR),
            # the workspace
            (dict(ws="k", by=512 * 512), FW | GR | MA), (dict(ws="lse", by=0), FW | GR | MA), (dict(ws="dk", by=0), GR),
            # between the others' rows
            (dict(dv="dk", by=256), set()), (dict(dk="k", by=256), set()), (dict(out="v", by=256 + 512 * 997), FW),
            (dict(dk="q", by=512 * 3), set()), (dict(out="q", by=512 * 3), set())):
        a = _desc()
        at = _fill(a)
        by = change.pop("by", 0)
        for x, y in change.items():
            at[x] = at[y] + by
        got = {x for x, refused in _call_all(a, at, n).items() if refused}
        assert got == want, (change, by, got)


@pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that are no memory: only where nothing can be launched")
def test_rows_of_the_cache_itself_are_refused_as_outputs():
    L = sk.lib()
    row, B, n, H, keep = 128, 2, 100, 2, 10
    names = ("k", "v", "mass", "k_out", "v_out", "mass_out", "index_out", "lengths_out", "ws")

    def refused(k_first=None, total=200, **kw):
        at = {x: (i + 1) << 36 for i, x in enumerate(names)}
        c = sk._CacheC(dtype=1, batch=B, heads=H, d=64, dv=64, len=n, keep=keep, first=1, recent=2, key_lengths=1 << 50)
        for x in ("k", "v", "k_out", "v_out"):
            setattr(c, x + "_stride", sk._i64x3(total * H * 64, H * 64, 64))
        if k_first is not None:
            at["k_out"] = at["k"] + k_first * H * row
        for x, (y, by) in kw.items():
            at[x] = at[y] + by
        code = L.sinkhorn_cache_evict(ctypes.byref(c), *[ctypes.c_void_p(at[x]) for x in names], 1 << 20, None)
        return code == sk.ERR_INVALID_ARG and any(x in L.sinkhorn_last_error() for x in (b"overlap", b"alias"))

    assert not refused()
    for first in (1, 50, 99):
        assert refused(first)
    assert not refused(100) and not refused(190)  # rows behind the cache, between its batch entries
    assert refused(191)  # its last row is the next entry's first
    for kw in (dict(v_out=("k", row)), dict(v_out=("k_out", 0)), dict(v_out=("k_out", row)), dict(k_out=("mass", 796)),
               dict(mass_out=("v", 0)), dict(index_out=("k_out", 0)), dict(lengths_out=("v", 8)), dict(ws=("mass", 0)),
               dict(ws=("k_out", 16))):
        assert refused(**kw), kw
    assert not refused(mass_out=("v", n * H * row))  # behind the first entry


def _side_calls():
    """Every entry point and its fp32 side arguments."""
    q, k, v = _qkv()
    out, lse = torch.zeros(2, 3, 4, 8, dtype=BF), torch.zeros(2, 4, 3)
    mass, w = torch.zeros(2, 2, 5), torch.ones(2, 3)
    bias = torch.zeros(2, 5)
    return [
        (sk.cross_attention, dict(q=q, k=k, v=v, key_bias=bias, row_weight=w, mass_in=mass, mass_out=mass.clone(),
                                  out=out, lse=lse)),
        (sk.cross_attention_grad, dict(dout=out, q=q, k=k, v=v, out=out.clone(), lse=lse, key_bias=bias, dq=q.clone(),
                                       dk=k.clone(), dv=v.clone())),
        (sk.attention_mass, dict(q=q, k=k, lse=lse, key_bias=bias, row_weight=w, mass_in=mass, mass_out=mass.clone())),
        (sk.cache_evict, dict(k=k, v=v, mass=mass, keep=3, k_out=k[:, :3].clone(), v_out=v[:, :3].clone(),
                              mass_out=mass[..., :3].clone())),
    ]


@pytest.mark.parametrize("call,name", [(i, n) for i, (_, kw) in enumerate(_side_calls()) for n, t in kw.items()
                                       if isinstance(t, torch.Tensor)])
def test_gradients_are_not_lost_silently(call, name):
    """What requires grad is refused in every place while a graph is recorded,
    and gets past that check otherwise (to the one of the device)."""
    fn, kw = _side_calls()[call]
    kw[name] = kw[name].detach().clone().requires_grad_()
    with pytest.raises(ValueError, match="grad"):
        fn(**kw)
    with torch.no_grad(), pytest.raises(ValueError, match="device tensors"):
        fn(**kw)


@pytest.mark.parametrize("call,name", [(i, n) for i, (_, kw) in enumerate(_side_calls()) for n, t in kw.items()
                                       if isinstance(t, torch.Tensor)])
def test_tangents_are_not_lost_silently(call, name):
    """Forward-mode tensors are refused in every place; others inside a dual
    level are not."""
    import torch.autograd.forward_ad as fw

    fn, kw = _side_calls()[call]
    with fw.dual_level():
        with pytest.raises(ValueError, match="device tensors"):
            fn(**kw)
        kw[name] = fw.make_dual(kw[name].detach().clone(), torch.ones_like(kw[name]))
        with pytest.raises(ValueError, match="tangent"):
            fn(**kw)
        kw[name] = fw.unpack_dual(kw[name]).primal
        with pytest.raises(ValueError, match="device tensors"):
            fn(**kw)


def test_function_transforms_are_refused():
    q, k, v = _qkv(dtype=torch.float32)
    run = lambda x: sk.cross_attention(x, k, v)[0]  # noqa: E731
    with pytest.raises(ValueError, match="tangent"):
        torch.func.jvp(run, (q,), (torch.ones_like(q),))
    with pytest.raises(ValueError, match="requires grad"):
        torch.func.grad(lambda x: run(x).sum())(q)


@pytest.mark.parametrize("dtype,size", [(0, 4), (1, 2), (2, 2)])
def test_heads_far_apart_are_read_where_they_are(dtype, size):
    """[B, H, L, d] operands whose heads lie 256 MB apart: only rows of q and
    dout whose heads share a tile, and span 1 GB together, are copied. The lengths
    do not matter."""
    L = sk.lib()
    far, row = (1 << 28) // size, 64

    def need(what, hq, hkv, lq, lk, q_heads, k_heads):
        a = sk._AttentionC(dtype=dtype, batch=1, heads_q=hq, heads_kv=hkv, d=64, dv=64, len_q=lq, len_k=lk, scale=0.125)
        for n, s in (("q", q_heads), ("dout", q_heads), ("k", k_heads), ("v", k_heads)):
            setattr(a, n + "_stride", sk._i64x3(0, row, s))
        n = ctypes.c_int64()
        assert L.sinkhorn_attention_workspace(ctypes.byref(a), what, FAKE, FAKE, FAKE, FAKE, ctypes.byref(n)) == sk.OK
        return n.value

    for lq, lk in ((1000, 1000), (1000, 999), (1, 4000), (40, 70)):
        for what in range(4):
            rows = 2 if what == 2 else 1  # q, and dout in the backward pass
            for hq, hkv, copied in ((8, 8, 0), (8, 4, 0), (8, 2, rows), (8, 1, rows), (6, 2, 0)):
                near = need(what, hq, hkv, lq, lk, 64 * lq, 64 * lk)
                pad = -(-size * lq * hq * 64 // 256) * 256
                assert need(what, hq, hkv, lq, lk, far, far) == near + copied * pad, (what, hq, hkv, lq, lk)
