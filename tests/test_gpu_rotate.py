"""GPU parity of the rotary positions, head norms and their gradient against
plain 64-bit forms (tests/paged_ref.py, which also derives the tolerances)."""
import math
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from attention_ref import assert_close  # noqa: E402
from paged_ref import Rotation  # noqa: E402

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


def _view(t, layout):
    """The same values in another layout of memory."""
    B, L, H, d = t.shape
    if layout == "blhd":
        return t.clone()
    if layout == "bhld":
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    if layout == "half":  # one half of a wider projection
        w = torch.full((B, L, 2 * H, d), 7.0, dtype=t.dtype, device=t.device)
        w[:, :, H:] = t
        return w[:, :, H:]
    if layout == "odd":  # neither base nor rows aligned
        w = torch.full((B * L * H * (d + 3) + 1,), 7.0, dtype=t.dtype, device=t.device)
        x = w[1:].view(B, L, H, d + 3)[..., :d]
        x.copy_(t)
        return x
    raise ValueError(layout)


def _make(dtype, B, L, Hq, Hkv, d, seed=0, gain=1.0):
    gen = torch.Generator().manual_seed(seed)
    mk = lambda H: (gain * torch.randn(B, L, H, d, generator=gen)).to(dtype).to(DEV)  # noqa: E731
    return gen, mk(Hq), (mk(Hkv) if Hkv else None)


def _check(sk, q, k, what, q_out=None, k_out=None, **kw):
    B, L, _, d = q.shape
    common = dict(positions=kw.get("positions"), frequencies=kw.get("frequencies"), interleaved=kw.get("interleaved", False),
                  gain=kw.get("gain", 1.0), norm_eps=kw.get("norm_eps"), lengths=kw.get("lengths"), B=B, L=L, d=d)
    want = [(x, Rotation(q.dtype, weight=kw.get(n), **common).forward(x))
            for x, n in ((q, "q_weight"), (k, "k_weight")) if x is not None]
    got = sk.rotate_heads(q, k, q_out=q_out, k_out=k_out, **kw)
    for (_, (y, tol)), g, n in zip(want, got, "qk"):
        assert_close(g, y, tol, f"{what} {n}")
    return got


def _check_grad(sk, q, k, dq_out, dk_out, what, dq=None, dk=None, **kw):
    B, L, _, d = q.shape
    common = dict(positions=kw.get("positions"), frequencies=kw.get("frequencies"), interleaved=kw.get("interleaved", False),
                  gain=kw.get("gain", 1.0), norm_eps=kw.get("norm_eps"), lengths=kw.get("lengths"), B=B, L=L, d=d)
    refs = [Rotation(q.dtype, weight=kw.get(n), **common).grad(dy, x)
            for x, dy, n in ((q, dq_out, "q_weight"), (k, dk_out, "k_weight")) if x is not None]
    norm = kw.get("norm_eps") is not None
    got = sk.rotate_heads_grad(dq_out, dk_out, q if norm else None, k if norm else None, dq=dq, dk=dk, **kw)
    for i, ((dx, tol), w) in enumerate(refs):
        assert_close(got[i], dx, tol, f"{what} d{'qk'[i]}")
        if norm:
            assert_close(got[2 + i], w[0], w[1], f"{what} d{'qk'[i]}_weight")
        else:
            assert got[2 + i] is None
    return got


SHAPES = [
    # B, L, Hq, Hkv, d, rotated
    (2, 5, 8, 2, 128, 128),
    (4, 1, 8, 8, 64, 64),
    (1, 33, 3, 1, 64, 32),
    (2, 7, 5, 5, 80, 80),
    (1, 9, 4, 2, 72, 72),
    (3, 11, 2, 1, 50, 50),
    (2, 4, 4, 4, 50, 26),
    (1, 6, 3, 3, 33, 32),
    (1, 3, 2, 1, 1, 0),
    (1, 3, 2, 2, 2, 2),
    (2, 130, 6, 2, 128, 2),
    (1, 17, 1, 0, 96, 24),
    (1, 2, 70, 3, 96, 96),
    (1, 1, 1, 1, 127, 126),
    (3, 300, 1, 1, 32, 16),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "pairs"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_rotate_and_gradient(sk, dtype, interleaved, shape):
    B, L, Hq, Hkv, d, r = shape
    _log(f"rotate {dtype} {shape} {interleaved}")
    gen, q, k = _make(dtype, B, L, Hq, Hkv, d)
    _, dq, dk = _make(dtype, B, L, Hq, Hkv, d, seed=1)
    pos = torch.randint(-50, 100000, (B, L), generator=gen).int().to(DEV)
    f = sk.rotary_frequencies(r, device=DEV)
    kw = dict(positions=pos, frequencies=f, interleaved=interleaved, gain=1.3)
    _check(sk, q, k, "rotation", **kw)
    _check_grad(sk, q, k, dq, dk, "rotation", **kw)
    for wt in (F32, dtype):
        w = [(1 + 0.2 * torch.randn(d, generator=gen)).to(wt).to(DEV) for _ in range(2)]
        kw.update(norm_eps=1e-5, q_weight=w[0], k_weight=w[1] if Hkv else None)
        _check(sk, q, k, "norm", **kw)
        _check_grad(sk, q, k, dq, dk, "norm", **kw)
    _check(sk, q, k, "norm alone", norm_eps=1e-6)
    _check_grad(sk, q, k, dq, dk, "norm alone", norm_eps=1e-6)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("layout", ["blhd", "bhld", "half", "odd"])
@pytest.mark.parametrize("norm", [None, 1e-6])
def test_layouts_and_in_place(sk, dtype, layout, norm):
    _log(f"layouts {dtype} {layout} {norm}")
    gen, q, k = _make(dtype, 2, 9, 4, 2, 64)
    _, dq, dk = _make(dtype, 2, 9, 4, 2, 64, seed=1)
    kw = dict(frequencies=sk.rotary_frequencies(64, device=DEV), norm_eps=norm)
    V = [_view(t, layout) for t in (q, k, dq, dk)]
    # to the tolerances of the definition: unaligned rows are read in other chunks, whose
    # squares add up in another order
    want = _check(sk, V[0], V[1], "new outputs", **kw)
    gwant = _check_grad(sk, *V, "new outputs", **kw)
    out = [_view(torch.zeros_like(t), layout) for t in (q, k)]
    whole = [o._base if o._base is not None else o for o in out]
    before = [w.clone() for w in whole]
    _check(sk, V[0], V[1], "own outputs", q_out=out[0], k_out=out[1], **kw)
    for o, w, b in zip(out, whole, before):
        assert o.any()
        o.zero_()
        assert torch.equal(w, b)  # nothing beside it was written
    _check_grad(sk, *V, "own outputs", dq=out[0], dk=out[1], **kw)
    for o, w, b in zip(out, whole, before):
        assert o.any()
        o.zero_()
        assert torch.equal(w, b)
    # in place: the same chunks as into new outputs of this layout
    if layout != "odd":
        g = sk.rotate_heads_grad(V[2], V[3], V[0], V[1], dq=V[2], dk=V[3], **kw)
        assert g[0] is V[2] and torch.equal(V[2], gwant[0]) and torch.equal(V[3], gwant[1])
        r = sk.rotate_heads(V[0], V[1], q_out=V[0], k_out=V[1], **kw)
        assert r[0] is V[0] and torch.equal(V[0], want[0]) and torch.equal(V[1], want[1])
    else:
        keep = [t.clone() for t in V]
        _check_grad_in_place(sk, keep, V, kw)


def _check_grad_in_place(sk, keep, V, kw):
    """Unaligned: in place against the definition on the values that were there."""
    B, L, _, d = keep[0].shape
    R = lambda: Rotation(keep[0].dtype, None, kw["frequencies"], False, 1.0, kw["norm_eps"], None, None, B, L, d)  # noqa: E731
    sk.rotate_heads_grad(V[2], V[3], V[0], V[1], dq=V[2], dk=V[3], **kw)
    for i in (0, 1):
        (dx, tol), _ = R().grad(keep[2 + i], keep[i])
        assert_close(V[2 + i], dx, tol, f"gradient {i} in place")
    sk.rotate_heads(V[0], V[1], q_out=V[0], k_out=V[1], **kw)
    for i in (0, 1):
        y, tol = R().forward(keep[i])
        assert_close(V[i], y, tol, f"result {i} in place")


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("d", [50, 128])
def test_positions(sk, dtype, d):
    _log(f"positions {dtype} {d}")
    B, L = 2, 6
    gen, q, k = _make(dtype, B, L, 3, 1, d)
    f = sk.rotary_frequencies(d, base=500000.0, factor=8.0, original_length=8192, low=1.0, high=4.0, device=DEV)
    first = _check(sk, q, k, "default", frequencies=f)
    row = torch.arange(L, dtype=torch.int32, device=DEV)
    assert torch.equal(_check(sk, q, k, "one row", frequencies=f, positions=row)[0], first[0])
    far = torch.tensor([2 ** 31 - 1, -(2 ** 31), 2 ** 30 + 1, 1048575, 0, -1], dtype=torch.int32, device=DEV)
    _check(sk, q, k, "far", frequencies=f, positions=far)
    wide = torch.randint(0, 1 << 20, (B, 3 * L), generator=gen).int().to(DEV)
    _check(sk, q, k, "strided", frequencies=f, positions=wide[:, L:2 * L])
    _check(sk, q, k, "shared", frequencies=f, positions=row.view(1, L).expand(B, L))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("norm", [None, 1e-6])
def test_rows_behind_their_sequence(sk, dtype, bad, norm):
    _log(f"lengths {dtype} {bad} {norm}")
    B, L = 5, 9
    gen, q, k = _make(dtype, B, L, 4, 2, 64)
    _, dq, dk = _make(dtype, B, L, 4, 2, 64, seed=1)
    n = torch.tensor([9, 0, 4, 99, -3], dtype=torch.int32, device=DEV)
    kw = dict(frequencies=sk.rotary_frequencies(32, device=DEV), norm_eps=norm, lengths=n)
    clean = _check(sk, q, k, "clean", **kw), _check_grad(sk, q, k, dq, dk, "clean", **kw)
    for t in (q, k, dq, dk):
        for b, m in enumerate([9, 0, 4, 9, 0]):
            t[b, m:] = bad
    got = sk.rotate_heads(q, k, **kw), sk.rotate_heads_grad(dq, dk, q, k, **kw)
    for x, y in zip(got[0] + got[1], clean[0] + clean[1]):
        assert (x is None and y is None) or torch.equal(x, y)
    assert not got[0][0][1].any() and not got[0][0][2, 4:].any()


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "pairs"])
@pytest.mark.parametrize("d,r", [(64, 64), (64, 32), (50, 26), (80, 40)])
def test_no_number_stays_in_its_pair(sk, dtype, interleaved, d, r):
    _log(f"no number {dtype} {interleaved} {d} {r}")
    _, q, _ = _make(dtype, 1, d, 1, 0, d)
    clean = sk.rotate_heads(q, frequencies=sk.rotary_frequencies(r, device=DEV), interleaved=interleaved)[0]
    for bad in (math.nan, math.inf):
        x = q.clone()
        i = torch.arange(d)
        x[0, i, 0, i] = bad  # element i of row i
        y = sk.rotate_heads(x, frequencies=sk.rotary_frequencies(r, device=DEV), interleaved=interleaved)[0]
        for row in range(d):
            mates = {row}
            if row < r:
                mates.add((row ^ 1) if interleaved else (row + r // 2) % r)
            others = [c for c in range(d) if c not in mates]
            assert torch.equal(y[0, row, 0, others], clean[0, row, 0, others]), (row, bad)
            assert not torch.isfinite(y[0, row, 0, row])
    # elements behind the rotated part come through as they are
    assert torch.equal(clean[..., r:], q[..., r:])


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_no_rows(sk, dtype):
    f = sk.rotary_frequencies(64, device=DEV)
    for B, L in ((0, 4), (3, 0)):
        q = torch.zeros(B, L, 2, 64, dtype=dtype, device=DEV)
        out, _ = sk.rotate_heads(q, frequencies=f)
        assert out.shape == q.shape
        dq, dk, wq, wk = sk.rotate_heads_grad(q, q, q, q, frequencies=f, norm_eps=1e-6)
        assert dq.shape == q.shape and not wq.any() and not wk.any()


def test_many_tokens_and_heads_far_apart(sk):
    """More rows than one round of workgroups, with heads and rows more than 4 GB apart."""
    _log("many tokens")
    gen = torch.Generator(device=DEV).manual_seed(3)
    B, L, H, d = 1, 40000, 2, 128
    big = torch.empty((2, 3 << 30), dtype=torch.uint8, device=DEV).view(BF)  # 3 GB a row: heads
    x = big.as_strided((B, L, H, d), (0, d, big.stride(0), 1))
    x.copy_(torch.randn(B, L, H, d, generator=gen, device=DEV).to(BF))
    dy = torch.randn(B, L, H, d, generator=gen, device=DEV).to(BF)
    kw = dict(frequencies=sk.rotary_frequencies(d, device=DEV), norm_eps=1e-6)
    _check(sk, x, None, "far", **kw)
    _check_grad(sk, x, None, dy, None, "far", **kw)


def test_gradient_against_differences(sk):
    """fp32 gradient of sum(result * c) against central differences in 64 bits."""
    _log("differences")
    B, L, H, d, r = 1, 2, 2, 12, 8
    gen, q, _ = _make(F32, B, L, H, 0, d)
    c = torch.randn(B, L, H, d, generator=gen).to(DEV)
    w = (1 + 0.2 * torch.randn(d, generator=gen)).to(DEV)
    f = sk.rotary_frequencies(r, device=DEV)
    for inter in (False, True):
        kw = dict(frequencies=f, interleaved=inter, gain=0.7, norm_eps=1e-3)
        dx, _, dw, _ = sk.rotate_heads_grad(c, None, q, None, q_weight=w, **kw)

        def loss(x, wt):
            R = Rotation(F32, None, f, inter, 0.7, 1e-3, wt, None, B, L, d)
            n, e, _ = R._norm(x)
            from paged_ref import turn
            return float((turn(n, e, R.a, 0.7, inter)[0] * c.cpu().double()).sum())

        x0, w0, h = q.cpu().double(), w.cpu().double(), 1e-5
        # a central difference is off by h^2 / 6 of a third derivative (of size 1e3 at most
        # here) and 2^-52 / h of the loss: below 1e-6
        for grad, base, which in ((dx, x0, 0), (dw, w0, 1)):
            for i in range(base.numel()):
                lo, hi = base.clone(), base.clone()
                lo.view(-1)[i] -= h
                hi.view(-1)[i] += h
                num = (loss(hi, w0) - loss(lo, w0)) / (2 * h) if which == 0 else (loss(x0, hi) - loss(x0, lo)) / (2 * h)
                assert abs(float(grad.reshape(-1)[i]) - num) <= 1e-5 * (1 + abs(num)), (which, i)


def test_graph_streams_and_repeats(sk):
    """A captured step replays with the eager bits, on a stream of its own, while another runs."""
    _log("graph")
    gen, q, k = _make(BF, 2, 64, 8, 2, 128)
    _, dq, dk = _make(BF, 2, 64, 8, 2, 128, seed=1)
    f = sk.rotary_frequencies(128, device=DEV)
    w = torch.ones(128, device=DEV)
    kw = dict(frequencies=f, norm_eps=1e-6, q_weight=w, k_weight=w)
    step = lambda: sk.rotate_heads(q, k, **kw) + sk.rotate_heads_grad(dq, dk, q, k, **kw)  # noqa: E731
    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step()
    for _ in range(3):
        for t in res:
            t.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(res, want))
        q.copy_(q.roll(1, 0))
        k.copy_(k.roll(1, 0))
        dq.copy_(dq.roll(1, 0))
        dk.copy_(dk.roll(1, 0))
        want = [t.clone() for t in step()]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "pairs"])
def test_calls_beyond_the_last_cache(sk, dtype, interleaved):
    """More than 256 MB in a call (results go past the caches) as in parts: the same bits."""
    _log(f"beyond the cache {dtype} {interleaved}")
    B, L, H, d = 4, (6000 if dtype != torch.float32 else 3000), 24, 128
    gen = torch.Generator(device=DEV).manual_seed(3)
    q, k, dq, dk = (torch.randn(B, L, h, d, generator=gen, device=DEV).to(dtype) for h in (H, 8, H, 8))
    kw = dict(frequencies=sk.rotary_frequencies(96, device=DEV), interleaved=interleaved, norm_eps=1e-6)
    assert 2 * q.numel() * q.element_size() > 1 << 28 > 3 * (q[0].numel() + k[0].numel()) * q.element_size()
    got, grads = sk.rotate_heads(q, k, **kw), sk.rotate_heads_grad(dq, dk, q, k, **kw)
    plain = sk.rotate_heads(q, k, frequencies=kw["frequencies"], interleaved=interleaved)
    for b in range(B):
        part = [x[b:b + 1] for x in (q, k, dq, dk)]
        for x, y in zip(got, sk.rotate_heads(*part[:2], **kw)):
            assert torch.equal(x[b:b + 1], y)
        for x, y in zip(grads[:2], sk.rotate_heads_grad(part[2], part[3], part[0], part[1], **kw)[:2]):
            assert torch.equal(x[b:b + 1], y)
        for x, y in zip(plain, sk.rotate_heads(*part[:2], frequencies=kw["frequencies"], interleaved=interleaved)):
            assert torch.equal(x[b:b + 1], y)
