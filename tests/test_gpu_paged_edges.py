"""Edges of decoding over a paged cache: rows that share a wave, far memory, what lies
around the places that are written, and the contiguous cache's operators beside the
paged ones. References and tolerances as in tests/paged_ref.py."""
import math
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from attention_ref import assert_close  # noqa: E402
from paged_ref import PagedRef, table_of  # noqa: E402

DEV = "cuda:0"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
DTYPES, IDS = [BF, HF, F32], ["bf16", "fp16", "fp32"]


@pytest.fixture(scope="module")
def sk():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import log_domain_sinkhorn_amd as sk

    return sk


def _log(msg):
    print(msg, file=sys.stderr, flush=True)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _make(dtype, lens, m, Hq, H, d, size, seed, extra=0):
    """(q, k_cache, v_cache, table, lengths), every slot of every page a number."""
    gen = torch.Generator().manual_seed(seed)
    pages = sum((n + size - 1) // size for n in lens) + 1
    table = table_of(lens, size, pages, gen, extra=extra)
    mk = lambda *s: torch.randn(*s, generator=gen).to(dtype).to(DEV)  # noqa: E731
    return [mk(len(lens), m, Hq, d), mk(pages, size, H, d), mk(pages, size, H, d), table.to(DEV), _ints(lens)]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("m,lens", [(3, [70, 3]), (16, [500, 40]), (40, [200, 64]), (130, [257, 130])])
@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("window", [{}, {"recent": 9, "first": 2}])
def test_rows_of_a_wave_are_independent(sk, dtype, m, lens, d, window):
    """A key that a row does not see has no influence on it, to the bit, however large the
    scores are that it gives others; rows that see it are off by their own roundings."""
    _log(f"independent {dtype} {m} {lens} {d} {window}")
    args = _make(dtype, lens, m, 4, 2, d, 16, seed=m + d)
    out, lse = sk.paged_attention(*args, **window)
    for size in (1e1, 1e3, math.inf):
        for b, n in enumerate(lens):
            for j in sorted({0, n - m, n - m // 2 - 1, n - 1}):
                x = args[1].clone()
                at = int(args[3][b, j // 16]), j % 16
                x[at][0] = size * args[0][b, -1, 0].sign()  # key head 0, towards a query that sees it
                o, z = sk.paged_attention(args[0], x, *args[2:], **window)
                p = torch.arange(n - m, n, device=DEV)
                see = p >= j
                if window:
                    see &= (j > p - window["recent"]) | (torch.tensor(j, device=DEV) < window["first"])
                changed = not torch.equal(z, lse)
                assert changed or not see.any(), (size, b, j)
                o[b, see, :2], z[b, :2, see] = out[b, see, :2], lse[b, :2, see]
                same = torch.equal(o, out), torch.equal(z, lse)
                assert same == (True, True), (size, b, j)


def test_written_tensors_raise_their_version(sk):
    """What a call writes of the caller's is marked as changed, what it reads is not."""
    _log("versions")
    B, L, H, d, size = 2, 4, 2, 32, 8
    mk = lambda *s: torch.randn(*s, device=DEV)  # noqa: E731
    q, k, v, y = (mk(B, L, H, d) for _ in range(4))
    f, table, have = sk.rotary_frequencies(d, device=DEV), _ints([[0, 1], [2, 3]]), _ints([5, 9])
    kc, vc = mk(4, size, H, d), mk(4, size, H, d)
    new = lambda *s, t=F32: torch.zeros(*s, dtype=t, device=DEV)  # noqa: E731
    I32 = torch.int32
    out, lse = sk.cross_attention(q, k, v)
    mass = mk(B, H, L).abs()
    P = sk.Problem(mk(9, 2), mk(7, 2), None, None, 1.0)
    g, rows = torch.zeros(7, device=DEV), torch.arange(3, device=DEV)
    f0 = P.halfstep_f(0.1, g)[0]
    calls = [
        (lambda o: sk.rotate_heads(q, k, frequencies=f, **o), dict(q_out=new(B, L, H, d), k_out=new(B, L, H, d)), (q, k)),
        (lambda o: sk.rotate_heads(o["q_out"], None, frequencies=f, q_out=o["q_out"]), dict(q_out=q.clone()), (f,)),
        (lambda o: sk.rotate_heads_grad(y, k, q, v, frequencies=f, norm_eps=1e-6, **o), dict(dq=new(B, L, H, d), dk=new(B, L, H, d)), (q, k, v, y)),
        (lambda o: sk.rotate_heads_grad(o["dq"], frequencies=f, dq=o["dq"]), dict(dq=y.clone()), (f,)),
        (lambda o: sk.cache_append(k, v, o["kc"], o["vc"], table, have, q=q, q_out=o["q"], lengths_out=o["n"], frequencies=f),
         dict(kc=kc.clone(), vc=vc.clone(), q=new(B, L, H, d), n=new(B, t=I32)), (q, k, v, table, have)),
        (lambda o: sk.paged_attention(q, kc, vc, table, have, **o), dict(out=new(B, L, H, d), lse=new(B, H, L)), (q, kc, vc)),
        (lambda o: sk.cross_attention(q, k, v, **o), dict(out=new(B, L, H, d), lse=new(B, H, L), mass_out=new(B, H, L)), (q, k, v)),
        (lambda o: sk.cross_attention_grad(y, q, k, v, out, lse, **o), {n: new(B, L, H, d) for n in ("dq", "dk", "dv")}, (q, k, v, y, out, lse)),
        (lambda o: sk.attention_mass(q, k, lse, **o), dict(mass_out=new(B, H, L)), (q, k, lse)),
        (lambda o: sk.cache_evict(k, v, mass, 3, **o), dict(k_out=new(B, 3, H, d), v_out=new(B, 3, H, d), mass_out=new(B, H, 3),
                                                            index_out=new(B, H, 3, t=I32), lengths_out=new(B, t=I32)), (k, v, mass)),
        (lambda o: P.halfstep_f(0.1, g, **o), dict(out=new(9)), (g,)),
        (lambda o: P.halfstep_g(0.1, f0, **o), dict(out=new(7)), (f0,)),
        (lambda o: P.solve(sk.Schedule(1.0, 0.5, fixed_iters=2), **o), dict(f=new(9), g=new(7)), ()),
        (lambda o: P.materialize_rows(0.1, f0, g, rows, **o), dict(T=new(3, 7), row_max=new(3)), (f0, g)),
        (lambda o: P.materialize_rows_noalloc(0.1, f0, g, rows, **o), dict(T=new(3, 7), row_max=new(3)), (f0, g)),
        (lambda o: P.barycentric(0.1, g, **o), dict(T=new(9, 2), grad=new(9, 2)), (g,)),
    ]
    for i, (call, outputs, inputs) in enumerate(calls):
        before, read = {n: t._version for n, t in outputs.items()}, [t._version for t in inputs]
        call(outputs)
        assert all(t._version > before[n] for n, t in outputs.items()), i
        assert [t._version for t in inputs] == read, i
    P.close()


def test_a_graph_that_saved_a_written_tensor_refuses(sk):
    """In place on an intermediate, without a graph: the backward pass that saved it raises
    instead of going on with other values."""
    _log("saved")
    f = sk.rotary_frequencies(32, device=DEV)
    x = torch.randn(3, 8, 4, 32, device=DEV, requires_grad=True)
    one, other = torch.ones(1, 1, 4, 32, device=DEV), torch.zeros(3, 8, 4, 32, device=DEV)
    for write in (lambda t: sk.rotate_heads(t, frequencies=f, q_out=t), lambda t: sk.rotate_heads_grad(t, frequencies=f, dq=t),
                  lambda t: sk.cache_append(one, one, t, other, _ints([[1]]), _ints([0]))):
        y = x * 2.0
        loss = (y * y).sum()
        with torch.no_grad():
            write(y)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()


@pytest.mark.parametrize("m", [1, 16, 40, 200])
@pytest.mark.parametrize("apart", [10.0, 16.0, 18.0, 20.0])
@pytest.mark.parametrize("at", [0, 300])
def test_many_small_weights_in_fp16(sk, m, apart, at):
    """One key takes nearly all of a row's weight and holds zeros; the result is what the
    thousands of others add up to, whose weights fp16 alone could not hold."""
    _log(f"small weights {m} {apart} {at}")
    n, d = 3000, 64
    gen = torch.Generator().manual_seed(22)
    q, kc, vc, table, _ = _make(HF, [n], m, 1, 1, d, 16, seed=22)
    q.zero_()
    q[..., 0] = 1.0
    kc.zero_()
    value = (64.0 + 64.0 * torch.rand(n, d, generator=gen)).to(HF)
    value[at] = 0.0
    ids = table[0, :(n + 15) // 16].long()
    places = torch.zeros(len(ids) * 16, 1, d, dtype=HF)
    places[:n, 0] = value
    vc[ids] = places.view(-1, 16, 1, d).to(DEV)
    kc[ids[at // 16], at % 16, 0, 0] = apart
    # the same for 4 x 64 heads: as many pairs as do not need their keys split
    kc, vc = (x.expand(-1, -1, 64, -1) for x in (kc, vc))
    out, lse = sk.paged_attention(q.expand(4, m, 64, d), kc, vc, table.expand(4, -1), _ints([n] * 4), scale=1.0)
    for x, axes in ((out, (0, 2)), (lse, (0, 1))):
        assert torch.equal(x, x.narrow(axes[0], 0, 1).narrow(axes[1], 0, 1).expand_as(x))
    v, E = value.double(), 2.0 ** -24
    for i in {0, m // 2, m - 1}:
        see = n - m + i + 1
        s = torch.zeros(see, dtype=torch.float64)
        s[at] = apart
        z = torch.logsumexp(s, 0)
        w = torch.exp(s - z)
        y, W = w @ v[:see], w @ v[:see].abs()
        # a held weight is off by half a step, 2^-11 of it or 2^-25 where it is small, and the
        # largest is held as 2^7 or more: 2^-32 of the sum. fp32: the score (one product), the
        # exponential and sums of `see` terms. The result is rounded once
        rel = E * (apart + 16 + see + 64)
        tol = (2.0 ** -11 * 1.01 + 2 * rel) * W + 2.0 ** -32 * 1.01 * v[:see].abs().sum(0) + 2.0 ** -11 * 1.01 * y.abs() + 2.0 ** -25
        assert_close(out[0, i, 0], y, tol, f"row {i}")
        assert abs(float(lse[0, 0, i]) - float(z)) <= rel + 4 * E * float(z) + 4 * E, i


def _far(t, axis):
    """t's values in memory where `axis` (of two places) lies 2^32 elements and a little apart."""
    shape, d = t.shape, t.shape[3]
    far, near = (1 << 32) + 8 * d, [0, 0, 0]
    n = d
    for a in (2, 1, 0):
        near[a] = far if a == axis else n
        n *= 1 if a == axis else shape[a]
    x = torch.empty(far + n, dtype=t.dtype, device=DEV).as_strided(shape, (*near, 1))
    x.copy_(t)
    assert torch.equal(x, t)
    return x


@pytest.mark.parametrize("axis", [0, 1, 2], ids=["sequences", "rows", "heads"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "pairs"])
def test_rotation_beyond_32_bits(sk, axis, interleaved):
    """Operands, results and gradients whose elements lie beyond 2^32, as in one piece."""
    _log(f"far {axis} {interleaved}")
    gen = torch.Generator().manual_seed(23)
    shape = [3, 3, 3, 128]
    shape[axis] = 2
    q, k, dq, dk = (torch.randn(shape, generator=gen).to(BF).to(DEV) for _ in range(4))
    kw = dict(frequencies=sk.rotary_frequencies(96, device=DEV), interleaved=interleaved)
    for norm in (None, 1e-6):
        kw["norm_eps"] = norm
        want, grads = sk.rotate_heads(q, k, **kw), sk.rotate_heads_grad(dq, dk, q, k, **kw)
        a, b = _far(q, axis), _far(torch.zeros_like(q), axis)
        got = sk.rotate_heads(a, k, q_out=b, **kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        got = sk.rotate_heads(q, a, k_out=b, **kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[0])
        c = _far(dq, axis)
        got = sk.rotate_heads_grad(c, dk, a, k, dq=b, **kw)
        assert all(torch.equal(x, y) for x, y in zip(got, grads) if y is not None)
        c.copy_(dk)
        a.copy_(k)
        got = sk.rotate_heads_grad(dq, c, q, a, dk=b, **kw)
        assert all(torch.equal(x, y) for x, y in zip(got, grads) if y is not None)
        del a, b, c


@pytest.mark.parametrize("axis", [0, 1, 2], ids=["sequences", "rows", "heads"])
def test_appending_from_beyond_32_bits(sk, axis):
    _log(f"append far {axis}")
    gen = torch.Generator().manual_seed(24)
    shape = [3, 3, 3, 128]
    shape[axis] = 2
    q, k, v = (torch.randn(shape, generator=gen).to(BF).to(DEV) for _ in range(3))
    B, L, H, d = shape
    table = torch.arange(B, dtype=torch.int32, device=DEV).view(B, 1)
    kw = dict(frequencies=sk.rotary_frequencies(d, device=DEV), norm_eps=1e-6)
    near, far = ([torch.zeros(B, 8, H, d, dtype=BF, device=DEV) for _ in range(2)] for _ in range(2))
    _, want = sk.cache_append(k, v, *near, table, _ints([2] * B), q=q, **kw)
    _, got = sk.cache_append(_far(k, axis), _far(v, axis), *far, table, _ints([2] * B), q=q, q_out=_far(torch.zeros_like(q), axis), **kw)
    assert torch.equal(got, want) and all(torch.equal(x, y) for x, y in zip(far, near))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("m", [1, 4, 50])
@pytest.mark.parametrize("window", [{}, {"recent": 20, "first": 3}])
def test_lengths_beyond_the_table(sk, dtype, m, window):
    """A length beyond the table's places is taken as their number, below 0 as none."""
    _log(f"beyond the table {dtype} {m} {window}")
    args = _make(dtype, [96, 96, 96, 96], m, 4, 2, 64, 16, seed=25)
    args[4] = _ints([2 ** 31 - 1, 97, -7, 95])
    out, lse = sk.paged_attention(*args, **window)
    ref = PagedRef(*args, **window)
    assert_close(out, ref.out, ref.out_tol, "out")
    assert_close(lse, ref.lse, ref.lse_tol, "lse")
    want = sk.paged_attention(*args[:4], _ints([96, 96, 0, 95]), **window)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("d,dv,r", [(50, 33, 26), (64, 128, 64), (80, 8, 40), (1, 1, 0), (127, 126, 126)])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "pairs"])
def test_appending_leaves_what_lies_around_a_row(sk, dtype, d, dv, r, interleaved):
    """Rows that start anywhere, with other data in front of, between and behind them."""
    _log(f"around {dtype} {d} {dv} {r}")
    gen = torch.Generator().manual_seed(26)
    pages, size, H, B, L = 6, 8, 3, 2, 11
    whole, views = [], []
    for w in (d, dv):
        t = torch.randn(pages * size * H * (w + 3) + 4, generator=gen).to(dtype).to(DEV)
        whole.append(t)
        views.append(t[1:-3].view(pages, size, H, w + 3)[..., :w])
    before = [t.clone() for t in whole]
    table = _ints([[4, 0, 7], [-1, 5, 2]])  # pages 1 and 3 are nobody's, 7 and -1 are none
    k, v, q = (torch.randn(B, L, H, w, generator=gen).to(dtype).to(DEV) for w in (d, dv, d))
    qw = torch.randn(B * L * H * (d + 3) + 4, generator=gen).to(dtype).to(DEV)
    qo, qb = qw[1:-3].view(B, L, H, d + 3)[..., :d], qw.clone()
    new = [9, 11]
    sk.cache_append(k, v, *views, table, _ints([3, 6]), new_lengths=_ints(new), q=q, q_out=qo, interleaved=interleaved, norm_eps=1e-6,
                    frequencies=sk.rotary_frequencies(r, device=DEV))
    places = [(4, s) for s in range(3, 8)] + [(0, s) for s in range(4)] + [(5, s) for s in range(8)] + [(2, 0)]
    for x, t, b in zip(views, whole, before):
        assert not torch.equal(t, b)
        old = b[1:-3].view(pages, size, H, -1)[..., :x.shape[3]]
        for at in places:
            x[at] = old[at]
        assert torch.equal(t, b)
    assert not torch.equal(qw, qb)
    qo.copy_(qb[1:-3].view(B, L, H, d + 3)[..., :d])
    assert torch.equal(qw, qb)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("new", [1, 5])
def test_evicted_cache_as_pages_of_one_sequence(sk, dtype, new):
    """The contiguous cache's operators and the paged ones together: keys are appended to a cache in
    one piece (a page a sequence), weighed and pruned; tokens that follow go behind those kept,
    at the positions they have in the text, and see all that is left."""
    _log(f"evicted {dtype} {new}")
    B, Hq, H, d, size, keep = 2, 4, 2, 64, 128, 40
    gen = torch.Generator().manual_seed(27)
    mk = lambda n, h: torch.randn(B, n, h, d, generator=gen).to(dtype).to(DEV)  # noqa: E731
    table, lens = torch.arange(B, dtype=torch.int32, device=DEV).view(B, 1), [100, 77]
    kw = dict(frequencies=sk.rotary_frequencies(d, device=DEV), norm_eps=1e-6)
    kc, vc, k2, v2 = (torch.zeros(B, size, H, d, dtype=dtype, device=DEV) for _ in range(4))
    have, q = sk.cache_append(mk(100, H), mk(100, H), kc, vc, table, _ints([0] * B), new_lengths=_ints(lens), q=mk(100, Hq), **kw)
    out, lse = sk.cross_attention(q[:, -1:], kc, vc, key_lengths=have)
    mass = sk.attention_mass(q[:, -1:], kc, lse, key_lengths=have)
    _, _, _, index, kept = sk.cache_evict(kc, vc, mass, keep, key_lengths=have, first=4, recent=8, k_out=k2[:, :keep], v_out=v2[:, :keep])
    assert kept.tolist() == [keep] * B
    for b in range(B):
        for h in range(H):
            at = index[b, h].long()
            assert torch.equal(k2[b, :keep, h], kc[b, at, h]) and torch.equal(v2[b, :keep, h], vc[b, at, h])
    k, v, x = mk(new, H), mk(new, H), mk(new, Hq)
    places = (have[:, None] + torch.arange(new, device=DEV)).int()  # in the text, not in the cache
    total, q = sk.cache_append(k, v, k2, v2, table, kept, positions=places, q=x, **kw)
    assert total.tolist() == [keep + new] * B
    qr, kr = sk.rotate_heads(x, k, positions=places, **kw)
    assert torch.equal(q, qr) and torch.equal(k2[:, keep:keep + new], kr) and torch.equal(v2[:, keep:keep + new], v)
    assert not k2[:, keep + new:].any() and not v2[:, keep + new:].any()
    got, z = sk.paged_attention(q, k2, v2, table, total)
    ref = PagedRef(q, k2, v2, table, total)
    assert_close(got, ref.out, ref.out_tol, "out")
    assert_close(z, ref.lse, ref.lse_tol, "lse")
    # the last token sees all keys, as in the contiguous operator
    o, y = sk.cross_attention(q[:, -1:], k2, v2, key_lengths=total)
    assert_close(o, ref.out[:, -1:], ref.out_tol[:, -1:], "contiguous out")
    assert_close(y, ref.lse[:, :, -1:], ref.lse_tol[:, :, -1:], "contiguous lse")
