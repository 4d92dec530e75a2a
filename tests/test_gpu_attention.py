"""GPU parity of cross attention, its gradient, the gathered weight and cache
eviction against plain 64-bit forms (tests/attention_ref.py, which also
derives the tolerances)."""
import math
import sys

import numpy as np
import pytest

import oracle
import synth

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from attention_ref import E, Ref, assert_close, evict_ref  # noqa: E402

DEV = "cuda:0"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
DTYPES = [BF, HF, F32]
IDS = ["bf16", "fp16", "fp32"]


@pytest.fixture(scope="module")
def sk():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import log_domain_sinkhorn_amd as sk

    return sk


def _log(msg):
    print(msg, file=sys.stderr, flush=True)


def _rand(gen, *shape, dtype=F32, gain=1.0):
    return (gain * torch.randn(*shape, generator=gen)).to(dtype).to(DEV)


def _view(t, layout):
    """The same values in another layout of memory."""
    B, L, H, d = t.shape
    if layout == "blhd":
        return t
    if layout == "bhld":
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    if layout == "half":  # one half of a wider projection
        w = torch.full((B, L, H, 2 * d), 7.0, dtype=t.dtype, device=t.device)
        w[..., d:] = t
        return w[..., d:]
    if layout == "odd":  # neither base nor rows aligned
        w = torch.full((B * L * H * (d + 3) + 1,), 7.0, dtype=t.dtype, device=t.device)
        x = w[1:].view(B, L, H, d + 3)[..., :d]
        x.copy_(t)
        return x
    raise ValueError(layout)


def _make(dtype, B, Lq, Hq, Hkv, Lk, d, dv, seed, layout="blhd", gain=1.0):
    gen = torch.Generator().manual_seed(seed)
    q = _view(_rand(gen, B, Lq, Hq, d, dtype=dtype, gain=gain), layout)
    k = _view(_rand(gen, B, Lk, Hkv, d, dtype=dtype), layout)
    v = _view(_rand(gen, B, Lk, Hkv, dv, dtype=dtype), layout)
    return gen, q, k, v


def _bias(gen, kind, B, Hkv, Lk):
    if kind is None:
        return None
    shape = (B, Hkv, Lk) if kind == "heads" else (B, Lk)
    x = torch.randn(*shape, generator=gen)
    drop = torch.rand(*shape, generator=gen)
    x[drop < 0.15] = -math.inf
    x[(drop >= 0.15) & (drop < 0.25)] = torch.finfo(F32).min
    return x.to(DEV)


def _check_forward(sk, q, k, v, what, **kw):
    out, lse = sk.cross_attention(q, k, v, **kw)
    kw = {x: y for x, y in kw.items() if x not in ("out", "lse")}
    ref = Ref(q, k, v, **kw)
    assert_close(lse, ref.lse, ref.lse_tol, what + " lse")
    assert_close(out, ref.out, ref.out_tol, what + " out")
    return out, lse, ref


SHAPES = [
    # B, Lq, Hq, Hkv, Lk, d, dv
    (1, 1, 1, 1, 1, 64, 64),
    (2, 1, 8, 2, 129, 128, 128),
    (3, 1, 4, 4, 1000, 64, 64),
    (1, 7, 6, 2, 2049, 80, 80),
    (2, 33, 2, 1, 65, 64, 32),
    (1, 128, 4, 4, 127, 128, 128),
    (2, 130, 3, 3, 300, 50, 50),
    (1, 200, 2, 2, 1, 8, 8),
    (1, 3, 1, 1, 31, 1, 1),
    (2, 40, 5, 1, 96, 72, 128),
    (1, 257, 1, 1, 513, 33, 7),
    (1, 64, 16, 1, 64, 96, 96),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward(sk, dtype, shape):
    _log(f"forward {dtype} {shape}")
    gen, q, k, v = _make(dtype, *shape, seed=1)
    _check_forward(sk, q, k, v, "plain")
    bias = _bias(gen, "shared", shape[0], shape[3], shape[4])
    _check_forward(sk, q, k, v, "bias", key_bias=bias, scale=0.3)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("layout", ["bhld", "half", "odd"])
@pytest.mark.parametrize("Lq", [1, 70])
def test_forward_layouts(sk, dtype, layout, Lq):
    _log(f"layouts {dtype} {layout} {Lq}")
    gen, q, k, v = _make(dtype, 2, Lq, 4, 2, 150, 64, 64, seed=2, layout=layout)
    ref = _check_forward(sk, q, k, v, layout)[2]
    # outputs in the caller's layout, and nothing beside them written
    out = _view(torch.zeros(2, Lq, 4, 64, dtype=dtype, device=DEV), layout)
    whole = out._base if out._base is not None else out
    before = whole.clone()
    sk.cross_attention(q, k, v, out=out)
    assert_close(out, ref.out, ref.out_tol, "out")
    got = whole.clone()
    out.zero_()
    assert torch.equal(whole, before) and not torch.equal(got, before)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("Lq", [1, 50])
def test_forward_lengths_and_head_bias(sk, dtype, Lq):
    _log(f"lengths {dtype} {Lq}")
    B, Hq, Hkv, Lk, d = 5, 4, 2, 333, 64
    gen, q, k, v = _make(dtype, B, Lq, Hq, Hkv, Lk, d, d, seed=3)
    klen = torch.tensor([333, 0, 1, 64, 999], dtype=torch.int32, device=DEV)
    qlen = torch.tensor([Lq, Lq, 0, (Lq + 1) // 2, -3], dtype=torch.int32, device=DEV)
    bias = _bias(gen, "heads", B, Hkv, Lk)
    _check_forward(sk, q, k, v, "keys", key_lengths=klen)
    _check_forward(sk, q, k, v, "both", key_lengths=klen, query_lengths=qlen)
    out, lse, _ = _check_forward(sk, q, k, v, "all", key_lengths=klen, query_lengths=qlen, key_bias=bias)
    assert float(out[1].abs().max()) == 0.0 and bool((lse[1] == -math.inf).all())


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("Lq", [2, 45])
@pytest.mark.parametrize("poison", [math.nan, math.inf, -math.inf])
def test_masked_places_may_hold_anything(sk, dtype, Lq, poison):
    _log(f"poison {dtype} {Lq} {poison}")
    B, Hq, Hkv, Lk, d = 2, 4, 2, 200, 64
    gen, q, k, v = _make(dtype, B, Lq, Hq, Hkv, Lk, d, d, seed=4)
    dout = _rand(gen, B, Lq, Hq, d, dtype=dtype)
    klen = torch.tensor([150, 199], dtype=torch.int32, device=DEV)
    qlen = torch.tensor([Lq, Lq - 1], dtype=torch.int32, device=DEV)
    bias = torch.zeros(B, Lk, device=DEV)
    bias[0, ::3] = -math.inf
    bias[1, 5:90] = torch.finfo(F32).min
    kw = dict(key_lengths=klen, query_lengths=qlen, key_bias=bias)
    mass = torch.empty(B, Hkv, Lk, device=DEV)
    out, lse = sk.cross_attention(q, k, v, mass_out=mass, **kw)
    grads = sk.cross_attention_grad(dout, q, k, v, out, lse, **kw)
    q2, k2, v2, d2, b2 = q.clone(), k.clone(), v.clone(), dout.clone(), bias.clone()
    q2[1, Lq - 1:] = poison
    d2[1, Lq - 1:] = poison
    for t in (k2, v2):
        t[0, 150:] = poison
        t[1, 199:] = poison
        t[0, ::3] = poison
        t[1, 5:90] = poison
    b2[0, 150:] = poison
    b2[1, 199:] = poison
    kw["key_bias"] = b2
    mass2 = torch.empty_like(mass)
    out2, lse2 = sk.cross_attention(q2, k2, v2, mass_out=mass2, **kw)
    assert torch.equal(out, out2) and torch.equal(lse, lse2) and torch.equal(mass, mass2)
    assert torch.equal(sk.attention_mass(q2, k2, lse2, **kw), sk.attention_mass(q, k, lse, **{**kw, "key_bias": bias}))
    o2, l2 = out2.clone(), lse2.clone()
    o2[1, Lq - 1:] = poison
    l2[1, :, Lq - 1:] = poison
    for a, b in zip(grads, sk.cross_attention_grad(d2, q2, k2, v2, o2, l2, **kw)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_all_keys_masked_and_no_keys(sk, dtype):
    gen, q, k, v = _make(dtype, 2, 20, 2, 2, 40, 64, 64, seed=5)
    dout = _rand(gen, 2, 20, 2, 64, dtype=dtype)
    for low in (-math.inf, torch.finfo(F32).min, -1e30):
        bias = torch.zeros(2, 40, device=DEV)
        bias[1] = low
        out, lse, _ = _check_forward(sk, q, k, v, "masked", key_bias=bias)
        assert float(out[1].abs().max()) == 0.0
        dq, dk, dv = sk.cross_attention_grad(dout, q, k, v, out, lse, key_bias=bias)
        for g in (dq, dk, dv):
            assert float(g[1].abs().max()) == 0.0 and bool(torch.isfinite(g).all())
    empty = k[:, :0]
    mass = torch.empty(2, 2, 0, device=DEV)
    out, lse = sk.cross_attention(q, empty, v[:, :0], mass_out=mass)
    assert float(out.abs().max()) == 0.0 and bool((lse == -math.inf).all())
    dq, dk, dv = sk.cross_attention_grad(dout, q, empty, v[:, :0], out, lse)
    assert float(dq.abs().max()) == 0.0 and dk.shape[1] == 0
    out, lse = sk.cross_attention(q[:, :0], k, v)
    assert out.shape == (2, 0, 2, 64) and lse.shape == (2, 2, 0)
    dq, dk, dv = sk.cross_attention_grad(dout[:, :0], q[:, :0], k, v, out, lse)
    assert float(dk.abs().max()) == 0.0 and float(dv.abs().max()) == 0.0
    mass = torch.rand(2, 2, 40, device=DEV)
    assert torch.equal(sk.attention_mass(q[:, :0], k, lse, mass_in=mass), mass)
    out, lse = sk.cross_attention(q[:0], k[:0], v[:0])
    assert out.shape[0] == 0


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_sharp_and_large_scores(sk, dtype):
    """Scores of hundreds with the maximum late, early and tied."""
    gen, q, k, v = _make(dtype, 1, 64, 2, 2, 700, 64, 64, seed=6, gain=8.0)
    k[:, -1] = 4.0 * q[:, 0, :, :].sign()
    k[:, 0] = -4.0 * q[:, 0, :, :].sign()
    k[:, 350] = k[:, 10]
    _check_forward(sk, q, k, v, "sharp", scale=0.5)
    bias = torch.full((1, 700), -65504.0, device=DEV)
    bias[0, 100:120] = 0.0
    _check_forward(sk, q, k, v, "lowest fp16", key_bias=bias, scale=0.05)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("shape", [(2, 1, 8, 2, 5000, 128, 64), (1, 5, 6, 1, 3001, 50, 50), (2, 32, 1, 1, 700, 64, 64),
                                   (1, 90, 4, 2, 1111, 64, 64), (1, 1, 1, 1, 1, 64, 64), (1, 300, 2, 2, 40, 80, 80)],
                         ids=lambda s: "x".join(map(str, s)))
def test_gathered_weight(sk, dtype, shape):
    _log(f"mass {dtype} {shape}")
    B, Lq, Hq, Hkv, Lk, d, dv = shape
    gen, q, k, v = _make(dtype, *shape, seed=7)
    mass = torch.rand(B, Hkv, Lk, generator=gen).to(DEV)
    w = torch.rand(B, Lq, generator=gen).to(DEV)
    klen = torch.randint(1, Lk + 1, (B,), generator=gen, dtype=torch.int32).to(DEV)
    bias = _bias(gen, "shared", B, Hkv, Lk)
    for kw in (dict(), dict(key_lengths=klen, key_bias=bias)):
        got = torch.empty_like(mass)
        out, lse = sk.cross_attention(q, k, v, row_weight=w, mass_in=mass, mass_out=got, **kw)
        ref = Ref(q, k, v, **kw)
        assert_close(out, ref.out, ref.out_tol, "out")
        assert_close(lse, ref.lse, ref.lse_tol, "lse")
        want, tol = ref.mass(mass, w)
        assert_close(got, want, tol, "fused weight")
        want, tol = Ref(q, k, lse=lse, **kw).mass(mass, w)
        assert_close(sk.attention_mass(q, k, lse, row_weight=w, mass_in=mass, **kw), want, tol, "own pass")
        want, tol = Ref(q, k, lse=lse, **kw).mass()
        assert_close(sk.attention_mass(q, k, lse, **kw), want, tol, "no start")
        acc = mass.clone()  # in place
        sk.cross_attention(q, k, v, row_weight=w, mass_in=acc, mass_out=acc, **kw)
        assert torch.equal(acc, got)


GRAD_SHAPES = [
    (1, 1, 1, 1, 1, 64, 64),
    (2, 33, 4, 2, 65, 64, 64),
    (1, 130, 2, 2, 129, 128, 128),
    (1, 50, 6, 1, 200, 50, 50),
    (2, 17, 2, 2, 300, 80, 64),
    (1, 300, 2, 1, 31, 33, 128),
    (1, 3, 1, 1, 40, 1, 5),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("layout", ["blhd", "half", "odd"])
@pytest.mark.parametrize("shape", GRAD_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_gradient(sk, dtype, shape, layout):
    _log(f"grad {dtype} {shape} {layout}")
    B, Lq, Hq, Hkv, Lk, d, dv = shape
    gen, q, k, v = _make(dtype, *shape, seed=8, layout=layout)
    dout = _view(_rand(gen, B, Lq, Hq, dv, dtype=dtype), layout)
    klen = torch.randint(1, Lk + 1, (B,), generator=gen, dtype=torch.int32).to(DEV)
    qlen = torch.randint(1, Lq + 1, (B,), generator=gen, dtype=torch.int32).to(DEV)
    bias = _bias(gen, "heads", B, Hkv, Lk)
    for kw in (dict(), dict(key_lengths=klen, query_lengths=qlen, key_bias=bias, scale=0.21)):
        out, lse = sk.cross_attention(q, k, v, **kw)
        grads = sk.cross_attention_grad(dout, q, k, v, out, lse, **kw)
        ref = Ref(q, k, v, lse=lse, **kw)
        for got, (want, tol), name in zip(grads, ref.grads(dout, out), ("dq", "dk", "dv")):
            assert got.dtype == dtype
            assert_close(got, want, tol, name)


@pytest.mark.parametrize("Lq,Lk", [(1, 4000), (4000, 5)])
def test_gradient_one_side_long(sk, Lq, Lk):
    """The streamed side split over workgroups."""
    gen, q, k, v = _make(F32, 1, Lq, 2, 1, Lk, 64, 64, seed=9)
    dout = _rand(gen, 1, Lq, 2, 64)
    out, lse = sk.cross_attention(q, k, v)
    ref = Ref(q, k, v, lse=lse)
    for got, (want, tol), name in zip(sk.cross_attention_grad(dout, q, k, v, out, lse), ref.grads(dout, out),
                                      ("dq", "dk", "dv")):
        assert_close(got, want, tol, name)


def test_gradient_against_differences(sk):
    """Central differences of the forward pass along random directions. The
    step's own error is what the same differences leave in 64 bits."""
    gen, q, k, v = _make(F32, 1, 9, 4, 2, 37, 16, 12, seed=10)
    dout = _rand(gen, 1, 9, 4, 12)
    bias = _bias(gen, "shared", 1, 2, 37)
    out, lse = sk.cross_attention(q, k, v, key_bias=bias)
    grads = sk.cross_attention_grad(dout, q, k, v, out, lse, key_bias=bias)
    h = 2.0 ** -6
    for which in range(3):
        for _ in range(3):
            t = torch.randn((q, k, v)[which].shape, generator=gen).to(DEV)
            t = torch.round(t * 64) / 64  # exact shifts
            vals, exact, noise = [], [], 0.0
            for sign in (1.0, -1.0):
                args = [q, k, v]
                args[which] = args[which] + sign * h * t
                o, _ = sk.cross_attention(*args, key_bias=bias)
                r = Ref(*args, key_bias=bias)
                vals.append(float((o.double() * dout.double()).sum()))
                exact.append(float((r.out * dout.cpu().double()).sum()))
                noise += float((r.out_tol * dout.cpu().double().abs()).sum())
            ref = Ref(q, k, v, key_bias=bias)
            want, tol = ref.grads(dout, out)[which]
            # out's own rounding inside D: |dS| moves by P |dout| out_tol
            along = float((grads[which].double() * t.double()).sum())
            along64 = float((ref.grads(dout, ref.out)[which][0] * t.cpu().double()).sum())
            diff, diff64 = (vals[0] - vals[1]) / (2 * h), (exact[0] - exact[1]) / (2 * h)
            slack = float((tol * t.cpu().double().abs()).sum())
            dD = float((ref.out_tol * dout.cpu().double().abs()).sum()) * float(t.abs().max()) * float(
                max(q.abs().max(), k.abs().max())) * ref.scale
            assert abs(diff - along) <= abs(diff64 - along64) + noise / (2 * h) + slack + dD


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("B,n,H,d,dv,keep,first,recent", [
    (2, 100, 3, 64, 64, 40, 4, 8), (1, 5000, 2, 128, 64, 777, 0, 0), (3, 37, 1, 50, 33, 36, 1, 35),
    (1, 1, 1, 8, 8, 1, 0, 0), (2, 64, 2, 64, 64, 64, 3, 3), (1, 300, 1, 1, 200, 10, 5, 5), (1, 2049, 2, 16, 16, 1, 0, 0),
    (2, 1500, 1, 72, 72, 1000, 1000, 0),
])
def test_evict(sk, dtype, B, n, H, d, dv, keep, first, recent):
    _log(f"evict {dtype} {(B, n, H, d, dv, keep, first, recent)}")
    gen = torch.Generator().manual_seed(11)
    k = _view(_rand(gen, B, n, H, d, dtype=dtype), "bhld")
    v = _rand(gen, B, n, H, dv, dtype=dtype)
    heavy = torch.exp(3 * torch.randn(B, H, n, generator=gen))
    ties = torch.randint(0, 3, (B, H, n), generator=gen).float()
    ties[ties == 0] = -0.0
    odd = heavy.clone()
    sel = torch.rand(B, H, n, generator=gen)
    odd[sel < 0.1], odd[sel > 0.9], odd[(sel > 0.5) & (sel < 0.6)] = math.nan, -math.inf, math.inf
    odd[(sel > 0.6) & (sel < 0.7)] *= -1
    klen = torch.randint(0, n + 1, (B,), generator=gen, dtype=torch.int32)
    klen[0] = n
    for mass in (heavy, ties, odd, torch.zeros_like(heavy)):
        for lens in (None, klen):
            m = mass.to(DEV)
            cap = min(keep, n)
            k_out = torch.full((B, H, cap, d), 5.0, dtype=dtype, device=DEV).transpose(1, 2)
            got = sk.cache_evict(k, v, m, keep, key_lengths=None if lens is None else lens.to(DEV), first=first,
                                 recent=recent, k_out=k_out)
            ko, vo, mo, idx, left = (t.cpu() for t in got)
            kept = evict_ref(k, v, mass, keep, lens, first, recent)
            for b in range(B):
                for hh in range(H):
                    want = torch.from_numpy(kept[b][hh])
                    c = want.numel()
                    assert int(left[b]) == c
                    assert torch.equal(idx[b, hh, :c].long(), want)
                    assert torch.equal(ko[b, :c, hh], k.cpu()[b, want, hh])
                    assert torch.equal(vo[b, :c, hh], v.cpu()[b, want, hh])
                    assert torch.equal(mo[b, hh, :c].view(torch.int32), mass[b, hh, want].view(torch.int32))
                    assert bool((idx[b, hh, c:] == -1).all()) and bool((mo[b, hh, c:] == 0).all())
                    assert bool((ko[b, c:, hh] == 5.0).all()) and bool((vo[b, c:, hh] == 0).all())


def test_evict_unaligned_rows_and_no_keys(sk):
    gen = torch.Generator().manual_seed(12)
    k = _view(_rand(gen, 2, 90, 2, 64, dtype=BF), "odd")
    v = _view(_rand(gen, 2, 90, 2, 64, dtype=BF), "half")
    mass = torch.rand(2, 2, 90, generator=gen)
    ko, vo, _, idx, _ = sk.cache_evict(k, v, mass.to(DEV), 30)
    kept = evict_ref(k, v, mass, 30)
    for b in range(2):
        for h in range(2):
            assert torch.equal(idx[b, h].cpu().long(), torch.from_numpy(kept[b][h]))
            assert torch.equal(ko[b, :, h], k[b, idx[b, h].long(), h])
            assert torch.equal(vo[b, :, h], v[b, idx[b, h].long(), h])
    out = sk.cache_evict(k[:, :0], v[:, :0], mass[..., :0].to(DEV), 30)
    assert out[0].shape[1] == 0 and out[4].tolist() == [0, 0]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_decode_evict_decode(sk, dtype):
    """A serving loop: tokens against cached states with the weight kept, an
    eviction, then a token against the pruned cache."""
    B, Hq, Hkv, Lk, d, keep = 2, 8, 2, 600, 64, 200
    gen, q, k, v = _make(dtype, B, 4, Hq, Hkv, Lk, d, d, seed=13, layout="bhld")
    klen = torch.tensor([600, 431], dtype=torch.int32, device=DEV)
    mass = torch.zeros(B, Hkv, Lk, device=DEV)
    want, tol = torch.zeros(B, Hkv, Lk, dtype=torch.float64), 0.0
    for i in range(3):
        sk.cross_attention(q[:, i:i + 1], k, v, key_lengths=klen, mass_in=mass, mass_out=mass)
        ref = Ref(q[:, i:i + 1], k, key_lengths=klen)
        x, t = ref.mass()
        want, tol = want + x, tol + t + 2 * E * (want + x)
    assert_close(mass, want, tol, "weight of three tokens")
    ko, vo, mo, idx, left = sk.cache_evict(k, v, mass, keep, key_lengths=klen, first=2, recent=20)
    kept = evict_ref(k, v, mass.cpu(), keep, klen.cpu(), 2, 20)
    out, lse = sk.cross_attention(q[:, 3:], ko, vo, key_lengths=left)
    for b in range(B):
        for h in range(Hkv):
            sel = torch.from_numpy(kept[b][h]).to(DEV)
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            ref = Ref(q[b:b + 1, 3:, heads], k[b:b + 1, sel, h:h + 1], v[b:b + 1, sel, h:h + 1])
            assert_close(out[b:b + 1, :, heads], ref.out, ref.out_tol, "pruned out")
            assert_close(lse[b:b + 1, heads], ref.lse, ref.lse_tol, "pruned lse")


def _as_attention(c, g, eps, scale):
    """Inputs of cross attention for plan rows of clouds c (centred: the
    projection moves with the clouds)."""
    mid = c.y.astype(np.float64).mean(0)
    x, y = c.x - mid, c.y - mid
    bias = np.log(np.maximum(c.b.astype(np.float64), 1e-300)) + (g - scale * (y * y).sum(1)) / eps
    f = lambda a: torch.from_numpy(np.ascontiguousarray(a.astype(np.float32))).to(DEV)  # noqa: E731
    return f(x)[None, :, None], f(y)[None, :, None], f(bias)[None], mid


@pytest.mark.parametrize("w,n,m,d,eps", [(2, 700, 900, 3, 0.05), (3, 500, 800, 50, 0.2)])
def test_barycentric_projection_and_column_marginal(sk, w, n, m, d, eps):
    """The transport plan through attention: the projection of its rows (here
    also for d = 50) and, with row weights a, its column marginal."""
    c = synth.make(w, n=n, m=m, **({"d": d} if w == 3 else {}))
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    scale = 1.0 if w == 2 else 1.0 / oracle.mean_sqeuclid(c.x, c.y)
    with sk.Problem(t(c.x), t(c.y), t(c.a), t(c.b), scale) as P:
        g = torch.zeros(m, device=DEV)
        for _ in range(4):
            f, _ = P.halfstep_f(eps, g)
            g, _ = P.halfstep_g(eps, f)
        f, _ = P.halfstep_f(eps, g)
        own = P.barycentric(eps, g, f_hint=f)[0] if d <= 8 else None
    gh = g.cpu().numpy().astype(np.float64)
    q, k, bias, mid = _as_attention(c, gh, eps, scale)
    mass = torch.empty(1, 1, m, device=DEV)
    out, lse = sk.cross_attention(q, k, k, scale=2 * scale / eps, key_bias=bias, row_weight=t(c.a)[None], mass_out=mass)
    ref = Ref(q, k, k, scale=2 * scale / eps, key_bias=bias)
    Tr = oracle.barycentric_rows(c.x, c.y, c.b, gh, eps, scale)
    T = out[0, :, 0].cpu().double() + torch.from_numpy(mid)
    # the call's own error, plus the rounding of its fp32 inputs (bias, centred points) into the scores
    mag = float(bias[bias > -1e30].abs().max()) + 2 * float(ref.dw.max()) / E
    slack = ref.out_tol[0, :, 0] + 4 * E * mag * float(k.abs().max())
    assert bool(((T - torch.from_numpy(Tr)).abs() <= slack).all())
    if own is not None:
        assert bool(((own.cpu().double() - T).abs() <= slack + 1e-5 * (1 + T.abs())).all())
    # f is the f-step of g, so pi_ij = a_i softmax_ij and the column marginal is the gathered weight
    C = scale * ((c.x[:, None, :].astype(np.float64) - c.y[None].astype(np.float64)) ** 2).sum(2)
    fr = oracle.halfstep_f(c.x, c.y, c.b, gh, eps, scale)
    pi = c.a[:, None].astype(np.float64) * c.b[None].astype(np.float64) * np.exp((fr[:, None] + gh[None] - C) / eps)
    want = torch.from_numpy(pi.sum(0))[None, None]
    _, tol = ref.mass(None, t(c.a)[None])
    assert_close(mass, want, tol + 4 * E * mag * want, "column marginal")


def test_results_repeat_bit_for_bit(sk):
    for shape in ((2, 1, 8, 2, 3000, 64, 64), (2, 100, 4, 2, 500, 128, 128)):
        gen, q, k, v = _make(BF, *shape, seed=14)
        dout = _rand(gen, shape[0], shape[1], shape[2], shape[6], dtype=BF)
        first = None
        for _ in range(3):
            mass = torch.empty(shape[0], shape[3], shape[4], device=DEV)
            out, lse = sk.cross_attention(q, k, v, mass_out=mass)
            res = (out, lse, mass, sk.attention_mass(q, k, lse)) + sk.cross_attention_grad(dout, q, k, v, out, lse)
            if first is None:
                first = [t.clone() for t in res]
            assert all(torch.equal(a, b) for a, b in zip(first, res))


def test_broadcast_inputs(sk):
    """One set of states shared by a batch (stride 0), and a gradient of out
    that is one number everywhere."""
    gen, q, k, v = _make(F32, 3, 20, 4, 2, 50, 64, 64, seed=15)
    k, v = k[:1].expand(3, -1, -1, -1), v[:1].expand(3, -1, -1, -1)
    out, lse, ref = _check_forward(sk, q, k, v, "shared states")
    dout = torch.tensor(0.5, device=DEV).expand(out.shape[0], 20, 4, 1).expand(3, 20, 4, 64)
    with pytest.raises(ValueError):
        sk.cross_attention_grad(dout, q, k, v, out, lse)  # its last dimension is no run of memory
    row = torch.randn(64, generator=gen).to(DEV).expand(3, 20, 4, 64)
    ref = Ref(q, k, v, lse=lse)
    for got, (want, tol), name in zip(sk.cross_attention_grad(row, q, k, v, out, lse), ref.grads(row, out),
                                      ("dq", "dk", "dv")):
        assert_close(got, want, tol, name)
    with pytest.raises(ValueError):
        sk.cross_attention(q, k, v, out=torch.empty(1, 20, 4, 64, device=DEV).expand(3, -1, -1, -1))


def test_side_stream(sk):
    gen, q, k, v = _make(HF, 2, 1, 8, 2, 4000, 64, 64, seed=16)
    want = sk.cross_attention(q, k, v)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        big = torch.randn(4096, 4096, device=DEV)
        for _ in range(4):
            big = big @ big * 1e-2
        k2 = k * 1.0  # made on the side stream, behind the work above
        got = sk.cross_attention(q, k2, v)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_graphs_replay(sk):
    """Two captured graphs (decode with weight and eviction; training step),
    replayed in turn with eager calls of the same operators between them."""
    B, Hq, Hkv, Lk, d, keep = 2, 8, 2, 700, 64, 128
    gen, q, k, v = _make(BF, B, 1, Hq, Hkv, Lk, d, d, seed=17)
    gen, q2, k2, v2 = _make(BF, B, 70, Hq, Hkv, 90, d, d, seed=18)
    dout = _rand(gen, B, 70, Hq, d, dtype=BF)
    klen = torch.tensor([700, 650], dtype=torch.int32, device=DEV)
    mass = torch.empty(B, Hkv, Lk, device=DEV)

    def decode():
        out, lse = sk.cross_attention(q, k, v, key_lengths=klen, mass_out=mass)
        return (out, lse, mass) + sk.cache_evict(k, v, mass, keep, key_lengths=klen, recent=8)

    def train():
        out, lse = sk.cross_attention(q2, k2, v2)
        return (out, lse) + sk.cross_attention_grad(dout, q2, k2, v2, out, lse)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        decode(), train()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for fn in (decode, train):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = fn()
        graphs.append((g, res, fn))
    for i in range(4):
        q.copy_(_rand(gen, B, 1, Hq, d, dtype=BF))
        q2.copy_(_rand(gen, B, 70, Hq, d, dtype=BF))
        for g, _, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        got = [[t.clone() for t in res] for _, res, _ in graphs]
        for (_, _, fn), r in zip(graphs, got):
            for a, b in zip(fn(), r):
                assert torch.equal(a, b), i
        torch.cuda.synchronize()


def test_cache_past_32_bit_offsets(sk):
    """A cache of more than 2^32 bytes and 2^31 elements: one batch entry's
    keys lie behind both borders."""
    H, d = 8, 128
    L = (1 << 21) + 77  # L * H * d > 2^31 elements
    _log("long cache")
    k = torch.zeros(1, L, H, d, dtype=BF, device=DEV)
    v = torch.zeros(1, L, H, d, dtype=BF, device=DEV)
    gen = torch.Generator().manual_seed(19)
    tail = 200
    k[:, -tail:] = _rand(gen, 1, tail, H, d, dtype=BF)
    v[:, -tail:] = _rand(gen, 1, tail, H, d, dtype=BF)
    q = _rand(gen, 1, 1, H, d, dtype=BF)
    bias = torch.full((1, L), -math.inf, device=DEV)
    bias[0, -tail:] = 0.0
    mass = torch.empty(1, H, L, device=DEV)
    out, lse = sk.cross_attention(q, k, v, key_bias=bias, mass_out=mass)
    ref = Ref(q, k[:, -tail:], v[:, -tail:])
    assert_close(out, ref.out, ref.out_tol, "out")
    want, tol = ref.mass()
    assert_close(mass[..., -tail:], want, tol, "weight")
    assert float(mass[..., :-tail].abs().max()) == 0.0
    ko, vo, mo, idx, left = sk.cache_evict(k, v, mass, 64)
    for h in range(H):
        sel = idx[0, h].long()
        assert bool((sel >= L - tail).all()) and torch.equal(ko[0, :, h], k[0, sel, h]) and torch.equal(vo[0, :, h], v[0, sel, h])


def test_wrong_arguments_are_refused(sk):
    gen, q, k, v = _make(BF, 2, 3, 4, 2, 10, 64, 64, seed=20)
    with pytest.raises(ValueError):
        sk.cross_attention(q, k, v, key_lengths=torch.ones(2, dtype=torch.int32))  # host lengths
    with pytest.raises(ValueError):
        sk.cross_attention(q, k.cpu(), v)
    with pytest.raises(sk.SinkhornError) as e:
        sk.cross_attention(q, k, v, out=q)
    assert e.value.code == sk.ERR_INVALID_ARG and "alias" in str(e.value)
    mass = torch.rand(2, 2, 10, device=DEV)
    with pytest.raises(sk.SinkhornError) as e:
        sk.cache_evict(k, v, mass, 10, k_out=k)
    assert e.value.code == sk.ERR_INVALID_ARG
    with pytest.raises(sk.SinkhornError) as e:
        sk.cache_evict(k, v, mass, 4, first=3, recent=2)
    assert "first + recent" in str(e.value)
