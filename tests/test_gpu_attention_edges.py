"""Cross attention, its gradient, the gathered weight and cache eviction where
their launch plans, tiles and loads change: head widths, groups and numbers of
heads, wide strides, long caches, values that are no numbers, two streams, and
shapes drawn at random. Plain forms and tolerances: tests/attention_ref.py."""
import math
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from attention_ref import Ref, assert_close, evict_ref  # noqa: E402

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


def _rand(gen, *shape, dtype=F32):
    return torch.randn(*shape, generator=gen).to(dtype).to(DEV)


def _check_all(sk, q, k, v, dout, what, weight=None, mass=None, **kw):
    """Every entry point on one set of inputs."""
    B, Lk, Hkv, _ = k.shape
    got = torch.empty(B, Hkv, Lk, device=DEV)
    out, lse = sk.cross_attention(q, k, v, row_weight=weight, mass_in=mass, mass_out=got, **kw)
    ref = Ref(q, k, v, **kw)
    assert_close(out, ref.out, ref.out_tol, what + " out")
    assert_close(lse, ref.lse, ref.lse_tol, what + " lse")
    assert_close(got, *ref.mass(mass, weight), what + " weight")
    o2, l2 = sk.cross_attention(q, k, v, **kw)
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    ref = Ref(q, k, v, lse=lse, **kw)
    assert_close(sk.attention_mass(q, k, lse, row_weight=weight, mass_in=mass, **kw), *ref.mass(mass, weight),
                 what + " own pass")
    for g, (want, tol), name in zip(sk.cross_attention_grad(dout, q, k, v, out, lse, **kw), ref.grads(dout, out),
                                    ("dq", "dk", "dv")):
        assert_close(g, want, tol, f"{what} {name}")


def _case(dtype, B, Lq, Hq, Hkv, Lk, d, dv, seed, ragged=True):
    gen = torch.Generator().manual_seed(seed)
    q, k = _rand(gen, B, Lq, Hq, d, dtype=dtype), _rand(gen, B, Lk, Hkv, d, dtype=dtype)
    v, dout = _rand(gen, B, Lk, Hkv, dv, dtype=dtype), _rand(gen, B, Lq, Hq, dv, dtype=dtype)
    kw = {}
    if ragged:
        bias = torch.randn(B, Lk, generator=gen)
        bias[torch.rand(B, Lk, generator=gen) < 0.2] = -math.inf
        kw = dict(key_bias=bias.to(DEV),
                  key_lengths=torch.randint(0, Lk + 1, (B,), generator=gen, dtype=torch.int32).to(DEV),
                  query_lengths=torch.randint(0, Lq + 1, (B,), generator=gen, dtype=torch.int32).to(DEV))
    extra = dict(weight=torch.rand(B, Lq, generator=gen).to(DEV), mass=torch.rand(B, Hkv, Lk, generator=gen).to(DEV))
    return (q, k, v, dout), kw, extra


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("d,dv", [(32, 24), (16, 32), (65, 96), (96, 80), (97, 1), (1, 128), (50, 50), (31, 63)])
def test_head_widths(sk, dtype, d, dv):
    for Lq in (1, 75):
        _log(f"widths {dtype} {d} {dv} {Lq}")
        args, kw, extra = _case(dtype, 2, Lq, 4, 2, 210, d, dv, seed=30)
        _check_all(sk, *args, f"Lq {Lq}", **kw, **extra)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("Lq,Hq,Hkv", [(60, 5, 1), (45, 6, 2), (20, 48, 1), (3, 96, 1), (11, 33, 1), (1, 40, 1), (1, 64, 2)])
def test_groups_across_tiles(sk, dtype, Lq, Hq, Hkv):
    """Query heads a key head that do not divide the tiles of rows, and more of
    them than a tile holds."""
    _log(f"groups {dtype} {Lq} {Hq} {Hkv}")
    args, kw, extra = _case(dtype, 2, Lq, Hq, Hkv, 140, 64, 64, seed=31)
    _check_all(sk, *args, "group", **kw, **extra)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("B,Hkv", [(13, 5), (8, 1), (3, 3), (64, 1), (9, 8), (70, 1)])
@pytest.mark.parametrize("Lq", [1, 36])
def test_numbers_of_heads(sk, dtype, B, Hkv, Lq):
    """Pairs of batch entry and key head: in eights, more than 64, fewer."""
    _log(f"pairs {dtype} {B} {Hkv} {Lq}")
    args, kw, extra = _case(dtype, B, Lq, Hkv, Hkv, 70, 64, 64, seed=32)
    _check_all(sk, *args, "pairs", **kw, **extra)


def _far(t, strides):
    """t at the given strides (elements) in a buffer of its own."""
    n = 1 + sum((s - 1) * x for s, x in zip(t.shape, strides))
    x = torch.empty(n, dtype=t.dtype, device=DEV).as_strided(t.shape, strides)
    x.copy_(t)
    return x


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("Lq", [1, 40])
def test_wide_strides(sk, dtype, Lq):
    """Rows 16 MB and heads more than 1 GB apart: a tile's offsets would pass
    31 bits."""
    _log(f"strides {dtype} {Lq}")
    (q, k, v, dout), kw, extra = _case(dtype, 1, Lq, 2, 1, 70, 64, 64, seed=33)
    row = (16 << 20) // q.element_size()
    want = sk.cross_attention(q, k, v, **kw)
    grads = sk.cross_attention_grad(dout, q, k, v, *want, **kw)
    far = lambda t: _far(t, (0, row, 64, 1))  # noqa: E731
    heads = lambda t: _far(t, (0, 64, (5 << 28) // t.element_size(), 1))  # noqa: E731
    for move in (far, heads):
        a = [move(q), move(k), move(v)]
        got = sk.cross_attention(*a, **kw)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        for x, y in zip(sk.cross_attention_grad(move(dout), *a, *got, **kw), grads):
            assert torch.equal(x, y)
        assert torch.equal(sk.attention_mass(a[0], a[1], got[1], **kw), sk.attention_mass(q, k, want[1], **kw))
    out = far(torch.zeros_like(want[0]))
    sk.cross_attention(q, k, v, out=out, **kw)
    assert torch.equal(out, want[0])


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_long_sequences_split(sk, dtype):
    """Keys split over workgroups with sequences of every length, and rows
    split over them in the backward pass."""
    for B, Lq, Hq, Hkv, Lk in ((4, 1, 8, 2, 9000), (4, 40, 2, 1, 5000), (2, 3000, 2, 1, 33)):
        _log(f"split {dtype} {B} {Lq} {Lk}")
        args, kw, extra = _case(dtype, B, Lq, Hq, Hkv, Lk, 64, 64, seed=34)
        kw["key_lengths"] = torch.tensor([Lk, 0, 1, Lk // 3][:B], dtype=torch.int32, device=DEV)
        kw["query_lengths"] = torch.tensor([Lq, Lq, Lq, Lq - 1][:B], dtype=torch.int32, device=DEV)
        _check_all(sk, *args, "split", **kw, **extra)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("Lq", [1, 50])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_live_values_that_are_no_numbers(sk, dtype, Lq, bad):
    """What a live key or row holds reaches its own results and no others."""
    (q, k, v, dout), _, _ = _case(dtype, 2, Lq, 4, 2, 150, 64, 64, seed=35, ragged=False)
    good = sk.cross_attention(q, k, v)
    k2 = k.clone()
    k2[1, 70, 1] = math.nan  # every row of batch entry 1, heads 2 and 3
    out, lse = sk.cross_attention(q, k2, v)
    assert bool(torch.isnan(out[1, :, 2:]).all()) and bool(torch.isnan(lse[1, 2:]).all())
    out[1, :, 2:], lse[1, 2:] = good[0][1, :, 2:], good[1][1, 2:]
    assert torch.equal(out, good[0]) and torch.equal(lse, good[1])
    v2 = v.clone()
    v2[0, 149, 0, 5] = bad  # one column of heads 0 and 1
    out, lse = sk.cross_attention(q, k, v2)
    assert not bool(torch.isfinite(out[0, :, :2, 5]).any())
    out[0, :, :2, 5] = good[0][0, :, :2, 5]
    assert torch.equal(out, good[0]) and torch.equal(lse, good[1])
    q2 = q.clone()
    q2[0, Lq - 1, 3] = math.nan
    out, lse = sk.cross_attention(q2, k, v)
    assert bool(torch.isnan(out[0, Lq - 1, 3]).all()) and bool(torch.isnan(lse[0, 3, Lq - 1]))
    out[0, Lq - 1, 3], lse[0, 3, Lq - 1] = good[0][0, Lq - 1, 3], good[1][0, 3, Lq - 1]
    assert torch.equal(out, good[0]) and torch.equal(lse, good[1])
    bias = torch.zeros(2, 150, device=DEV)
    bias[1, 3] = math.nan  # not masked: it reaches the whole entry
    out, lse = sk.cross_attention(q, k, v, key_bias=bias)
    assert bool(torch.isnan(out[1]).all()) and bool(torch.isfinite(out[0]).all())


@pytest.mark.parametrize("B,n,H,keep,first,recent", [
    (2, 4096, 3, 1024, 4, 128), (2, 4097, 1, 2000, 0, 9), (2, 16384, 1, 3000, 7, 100), (2, 20001, 2, 9000, 4, 64), (1, 65536, 1, 1, 0, 0), (2, 65537, 1, 30000, 0, 1),
    (1, 150001, 2, 149999, 11, 13), (3, 90000, 1, 40000, 40000, 0), (1, 70000, 1, 70000, 0, 0),
])
def test_evict_long(sk, B, n, H, keep, first, recent):
    """Each way of selecting: keys in registers, several a thread, streamed."""
    _log(f"evict {(B, n, H, keep, first, recent)}")
    gen = torch.Generator().manual_seed(36)
    k, v = _rand(gen, B, n, H, 8, dtype=BF), _rand(gen, B, n, H, 4, dtype=BF)
    heavy = torch.exp(3 * torch.randn(B, H, n, generator=gen))
    ties = torch.randint(0, 3, (B, H, n), generator=gen).float()
    ties[ties == 0] = -0.0
    sel = torch.rand(B, H, n, generator=gen)
    heavy2 = heavy.clone()
    heavy2[sel < 0.1], heavy2[sel > 0.9], heavy2[(sel > 0.5) & (sel < 0.6)] = math.nan, -math.inf, math.inf
    lens = torch.randint(0, n + 1, (B,), generator=gen, dtype=torch.int32)
    lens[-1] = n - 1
    for mass, ln in ((heavy, None), (ties, lens), (heavy2, lens), (torch.zeros_like(heavy), None)):
        got = sk.cache_evict(k, v, mass.to(DEV), keep, key_lengths=None if ln is None else ln.to(DEV), first=first,
                             recent=recent)
        ko, vo, mo, idx, left = (t.cpu() for t in got)
        kept = evict_ref(k, v, mass, keep, ln, first, recent)
        for b in range(B):
            for h in range(H):
                want = torch.from_numpy(kept[b][h])
                c = want.numel()
                assert int(left[b]) == c
                assert torch.equal(idx[b, h, :c].long(), want)
                assert torch.equal(ko[b, :c, h], k.cpu()[b, want, h]) and torch.equal(vo[b, :c, h], v.cpu()[b, want, h])
                assert torch.equal(mo[b, h, :c].view(torch.int32), mass[b, h, want].view(torch.int32))
                assert bool((idx[b, h, c:] == -1).all()) and bool((mo[b, h, c:] == 0).all())


def test_two_streams_at_once(sk):
    """Calls on two streams, each with its own workspace, do not meet."""
    cases = [_case(BF, 2, 1, 8, 2, 6000, 64, 64, seed=37), _case(BF, 2, 90, 8, 2, 400, 64, 64, seed=38)]

    def run(args, kw):
        q, k, v, dout = args
        mass = torch.empty(k.shape[0], k.shape[2], k.shape[1], device=DEV)
        out, lse = sk.cross_attention(q, k, v, mass_out=mass, **kw)
        return (out, lse, mass) + sk.cross_attention_grad(dout, q, k, v, out, lse, **kw) + tuple(
            sk.cache_evict(k, v, mass, 150, key_lengths=kw["key_lengths"], recent=4))

    want = [run(a, kw) for a, kw, _ in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(*cases[i][:2]))
    torch.cuda.synchronize()
    for w, rounds in zip(want, got):
        for r in rounds:
            # index_out and lengths are whole; rows behind a short sequence are zero from the binding
            assert all(torch.equal(x, y) for x, y in zip(w, r))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("seed", range(12))
def test_drawn_shapes(sk, dtype, seed):
    gen = torch.Generator().manual_seed(1000 + seed)
    pick = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=gen))  # noqa: E731
    Hkv, G, B = pick(1, 5), pick(1, 9), pick(1, 4)
    Lq = (1, pick(2, 8), pick(9, 200))[pick(0, 2)]
    Lk = (pick(1, 70), pick(71, 1500))[pick(0, 1)]
    d, dv = pick(1, 128), pick(1, 128)
    _log(f"drawn {dtype} {(B, Lq, Hkv * G, Hkv, Lk, d, dv)}")
    args, kw, extra = _case(dtype, B, Lq, Hkv * G, Hkv, Lk, d, dv, seed=2000 + seed, ragged=bool(seed % 3))
    _check_all(sk, *args, "drawn", **kw, **extra)


def test_evict_at_the_largest_length(sk):
    """2^31 - 1 keys, the most that are accepted: the places behind the kept
    keys, and a selection among keys up to the last one."""
    n = (1 << 31) - 1
    _log("evict 2^31 - 1, all places filled")
    row = torch.arange(1.0, 9.0, dtype=BF, device=DEV)
    k = row[:1].view(1, 1, 1, 1).expand(1, n, 1, 1)  # one row for all keys
    mass = torch.zeros(1, 1, n, device=DEV)
    guard = 4096
    index = torch.full((n + guard,), 7, dtype=torch.int32, device=DEV)
    weight = torch.full((n + guard,), 7.0, device=DEV)
    lens = torch.tensor([5], dtype=torch.int32, device=DEV)
    k_out, v_out = (torch.full((1, n, 1, 1), 3.0, dtype=BF, device=DEV) for _ in range(2))
    mass[0, 0, :6] = 2.0
    left = sk.cache_evict(k, k, mass, n, key_lengths=lens, k_out=k_out, v_out=v_out, mass_out=weight[:n].view(1, 1, n),
                          index_out=index[:n].view(1, 1, n))[4]
    assert left.tolist() == [5] and index[:5].tolist() == [0, 1, 2, 3, 4] and weight[:5].tolist() == [2.0] * 5
    assert int(index[5:n].max()) == -1 and int(index[5:n].min()) == -1
    assert float(weight[5:n].max()) == 0.0 and float(weight[5:n].min()) == 0.0
    assert bool((index[n:] == 7).all()) and bool((weight[n:] == 7.0).all())
    for t in (k_out, v_out):
        assert bool((t[0, :5] == 1.0).all()) and float(t[0, 5:].max()) == 3.0 and float(t[0, 5:].min()) == 3.0
    del index, weight, k_out, v_out
    _log("evict 2^31 - 1, selection")
    at = [0, 3, n // 2, n - 20000, n - 300, n - 2, n - 1]
    mass.zero_()
    mass[0, 0, at] = 1.0
    idx, left = sk.cache_evict(k, k, mass, 9)[3:]
    # the rest weigh nothing: the lowest indices
    assert left.tolist() == [9] and idx[0, 0].tolist() == sorted(at + [1, 2])


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("Lk", [90, 6000])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_weight_of_masked_keys_under_rows_that_are_no_numbers(sk, dtype, Lk, d, bad):
    """A key that takes no part gathers nothing, whatever a live row of q holds,
    in the fused form as in the pass of its own."""
    _log(f"masked weight {dtype} {Lk} {d} {bad}")
    for Lq in (1, 5, 40):
        (q, k, v, _), _, extra = _case(dtype, 2, Lq, 4, 2, Lk, d, d, seed=39, ragged=False)
        bias = torch.zeros(2, Lk, device=DEV)
        bias[:, ::3] = -math.inf
        bias[:, 1::7] = torch.finfo(F32).min
        lens = torch.tensor([Lk - 3, Lk - 40], dtype=torch.int32, device=DEV)
        masked = (bias < -1e29) | (torch.arange(Lk, device=DEV)[None] >= lens[:, None])
        masked = masked[:, None].expand(2, 2, Lk)
        q[:, Lq - 1, ::2, 5] = bad
        kw = dict(key_bias=bias, key_lengths=lens)
        got = torch.empty(2, 2, Lk, device=DEV)
        _, lse = sk.cross_attention(q, k, v, mass_in=extra["mass"], mass_out=got, **kw)
        own = sk.attention_mass(q, k, lse, mass_in=extra["mass"], **kw)
        for m in (got, own):
            assert torch.equal(m[masked], extra["mass"][masked])
            assert bool(torch.isnan(m[~masked]).all())


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("Lq", [1, 5, 40, 300])
@pytest.mark.parametrize("Lk", [70, 5000])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_without_keys_that_are_no_numbers(sk, dtype, Lq, Lk, d):
    """A row whose keys are all masked gives 0 and -infinity, whatever it holds,
    by its length as by its bias."""
    _log(f"rows without keys {dtype} {Lq} {Lk} {d}")
    (q, k, v, dout), _, _ = _case(dtype, 3, Lq, 4, 2, Lk, d, d, seed=40, ragged=False)
    bias = torch.zeros(3, 2, Lk, device=DEV)
    bias[1] = -math.inf  # entry 1 by its bias, of entry 2 the heads 2 and 3
    bias[2, 1] = torch.finfo(F32).min
    lens = torch.tensor([0, Lk, Lk - 1], dtype=torch.int32, device=DEV)
    kw = dict(key_bias=bias, key_lengths=lens)
    good = sk.cross_attention(q, k, v, **kw)
    for bad in (math.nan, math.inf, -math.inf):
        q2 = q.clone()
        q2[:2, Lq // 2:, :, 3] = bad
        q2[2, 0, 2:, d - 1] = bad
        got = torch.empty(3, 2, Lk, device=DEV)
        out, lse = sk.cross_attention(q2, k, v, mass_out=got, **kw)
        assert bool((out[:2] == 0).all()) and bool((lse[:2] == -math.inf).all())
        assert bool((out[2, :, 2:] == 0).all()) and bool((lse[2, 2:] == -math.inf).all())
        assert torch.equal(out, good[0]) and torch.equal(lse, good[1])
        assert bool((got[:2] == 0).all()) and bool((got[2, 1] == 0).all())


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("Lq,Lk", [(1, 70), (40, 300), (3, 5000)])
@pytest.mark.parametrize("d,dv", [(64, 64), (128, 80)])
def test_gradient_of_rows_without_keys_that_are_no_numbers(sk, dtype, Lq, Lk, d, dv):
    """No gradient of a row whose keys are all masked by bias, whatever q, dout
    and out hold there, and of its keys."""
    _log(f"gradient without keys {dtype} {Lq} {Lk} {d} {dv}")
    (q, k, v, dout), _, _ = _case(dtype, 2, Lq, 4, 2, Lk, d, dv, seed=41, ragged=False)
    bias = torch.zeros(2, 2, Lk, device=DEV)
    bias[1] = -math.inf
    bias[0, 1] = torch.finfo(F32).min
    kw = dict(key_bias=bias)
    out, lse = sk.cross_attention(q, k, v, **kw)
    good = sk.cross_attention_grad(dout, q, k, v, out, lse, **kw)
    for g in good:
        assert bool((g[1] == 0).all())
    for bad in (math.nan, math.inf):
        for which in range(3):
            args = [dout.clone(), q.clone(), k, v, out.clone(), lse]
            t = args[(0, 1, 4)[which]]
            t[1, Lq // 2:, :, 1] = bad
            t[0, 0, 2:, -1] = bad
            for got, want in zip(sk.cross_attention_grad(*args, **kw), good):
                assert torch.equal(got, want), (bad, which)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (4, 2), (3, 1)])
def test_heads_more_than_4_gb_apart(sk, dtype, Hq, Hkv):
    """Heads whose distance passes 32 bits, read where they are or (those that
    share a tile) from a copy."""
    _log(f"far heads {dtype} {Hq} {Hkv}")
    for Lq in (1, 90):
        (q, k, v, dout), kw, extra = _case(dtype, 1, Lq, Hq, Hkv, 70, 64, 64, seed=42)
        kw["query_lengths"] = None
        gap = ((1 << 32) + 4096) // q.element_size()
        far = lambda t: _far(t, (0, 64, gap, 1))  # noqa: E731
        q2, k2, v2, dout2 = far(q), far(k), far(v), far(dout)
        mass, mass2 = (torch.empty(1, Hkv, 70, device=DEV) for _ in range(2))
        want = sk.cross_attention(q, k, v, mass_out=mass, **kw)
        got = sk.cross_attention(q2, k2, v2, mass_out=mass2, **kw)
        assert all(torch.equal(x, y) for x, y in zip(got, want)) and torch.equal(mass, mass2)
        assert torch.equal(sk.attention_mass(q2, k2, got[1], **kw), sk.attention_mass(q, k, want[1], **kw))
        for x, y in zip(sk.cross_attention_grad(dout2, q2, k2, v2, *got, **kw),
                        sk.cross_attention_grad(dout, q, k, v, *want, **kw)):
            assert torch.equal(x, y)


@pytest.mark.parametrize("big", [(1 << 63) - 1, 1 << 63, (1 << 64) + 2, 1 << 100])
def test_evict_keeps_more_than_64_bits_count(sk, big):
    """A number of kept keys beyond 64 bits keeps all of them."""
    (_, k, v, _), _, extra = _case(BF, 2, 1, 4, 2, 50, 64, 64, seed=43, ragged=False)
    want = sk.cache_evict(k, v, extra["mass"], 50)
    for kw in (dict(), dict(first=3, recent=4), dict(first=big), dict(recent=big)):
        for got, x in zip(sk.cache_evict(k, v, extra["mass"], big, **kw), want):
            assert torch.equal(got, x)
    with pytest.raises(sk.SinkhornError):
        sk.cache_evict(k, v, extra["mass"], 10, first=big)
    with pytest.raises(sk.SinkhornError):
        sk.cache_evict(k, v, extra["mass"], 10, recent=-big)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("split", [False, True], ids=["whole", "split"])
def test_few_rows_over_many_tiles(sk, dtype, d, split):
    """Single tokens (and three) with the weight kept where a workgroup runs over
    nine tiles of live keys and more, alone on its keys or with others: the ring
    of tiles in its steady state."""
    size = torch.finfo(dtype).bits // 8
    keys = {128: 192, 256: 96, 512: 64}[size * (64 if d == 64 else 128)]  # of a tile
    # 256 pairs fill the compute units, with twelve tiles each; 32 are split in nine, nine tiles each
    B, Hkv, Lk, Lq, G = (16, 2, 79 * keys - 5, 1, 2) if split else (32, 8, 11 * keys + 7, 3, 1)
    _log(f"many tiles {dtype} {d} {(B, Hkv, Lk)}")
    (q, k, v, _), ragged, extra = _case(dtype, B, Lq, Hkv * G, Hkv, Lk, d, d, seed=44)
    ragged["key_lengths"][:3] = torch.tensor([Lk, Lk - 1, Lk - keys], dtype=torch.int32, device=DEV)
    for kw in (dict(), dict(key_bias=ragged["key_bias"]), ragged):
        got = torch.empty(B, Hkv, Lk, device=DEV)
        out, lse = sk.cross_attention(q, k, v, row_weight=extra["weight"], mass_in=extra["mass"], mass_out=got, **kw)
        o2, l2 = sk.cross_attention(q, k, v, **kw)
        assert torch.equal(out, o2) and torch.equal(lse, l2)
        ref = Ref(q, k, v, **kw)
        assert_close(out, ref.out, ref.out_tol, "out")
        assert_close(lse, ref.lse, ref.lse_tol, "lse")
        assert_close(got, *ref.mass(extra["mass"], extra["weight"]), "weight")


def _place(shape, dtype, layout):
    """(view, everything around it): room for an output in a layout of its own,
    filled with 7."""
    B, L, H, d = shape
    if layout == "heads":  # [B, H, L, d]
        x = torch.full((B, H, L, d), 7.0, dtype=dtype, device=DEV)
        return x.transpose(1, 2), x
    if layout == "half":  # one half of a wider projection
        x = torch.full((B, L, H, 2 * d), 7.0, dtype=dtype, device=DEV)
        return x[..., d:], x
    if layout == "odd":  # neither base nor rows aligned
        x = torch.full((B * L * H * (d + 3) + 1,), 7.0, dtype=dtype, device=DEV)
        return x[1:].view(B, L, H, d + 3)[..., :d], x
    x = torch.full((B, 2 * L, H, d), 7.0, dtype=dtype, device=DEV)  # behind other rows of each entry
    return x[:, L:], x


def _only(view, whole):
    """Nothing beside the view was written (the view itself is cleared)."""
    view.fill_(7.0)
    return bool((whole == 7.0).all())


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("layout", ["heads", "half", "odd", "behind"])
@pytest.mark.parametrize("shape", [(2, 33, 4, 2, 65, 64, 48), (1, 200, 4, 4, 300, 96, 128), (2, 3, 6, 2, 40, 40, 8),
                                   (1, 1, 2, 1, 4000, 64, 32), (1, 3000, 2, 1, 5, 32, 64)],
                         ids=lambda s: "x".join(map(str, s)))
def test_gradients_in_the_callers_tensors(sk, dtype, layout, shape):
    """dq, dk and dv of different widths in strided tensors, from whole and from
    split passes: the same bits as in new ones, and nothing beside them."""
    _log(f"own gradients {dtype} {layout} {shape}")
    (q, k, v, dout), kw, _ = _case(dtype, *shape, seed=45)
    out, lse = sk.cross_attention(q, k, v, **kw)
    want = sk.cross_attention_grad(dout, q, k, v, out, lse, **kw)
    own = [_place(t.shape, dtype, layout) for t in want]
    got = sk.cross_attention_grad(dout, q, k, v, out, lse, dq=own[0][0], dk=own[1][0], dv=own[2][0], **kw)
    for g, w, (view, whole) in zip(got, want, own):
        assert g.data_ptr() == view.data_ptr() and torch.equal(g, w)
    for view, whole in own:
        assert _only(view, whole)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_gradients_side_by_side(sk, dtype):
    """The gradients of one projection's parts (q, k and v of the same length) in
    the parts of one tensor, and out in the place behind them."""
    B, L, H, d = 2, 77, 3, 64
    gen = torch.Generator().manual_seed(46)
    qkv, dout = _rand(gen, B, L, 4, H, d, dtype=dtype), _rand(gen, B, L, H, d, dtype=dtype)
    q, k, v = qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]
    want = sk.cross_attention(q, k, v)
    out, lse = sk.cross_attention(q, k, v, out=qkv[:, :, 3])  # between the rows of its inputs
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    grads = sk.cross_attention_grad(dout, q, k, v, out, lse)
    whole = torch.full_like(qkv, 7.0)
    sk.cross_attention_grad(dout, q, k, v, out, lse, dq=whole[:, :, 0], dk=whole[:, :, 1], dv=whole[:, :, 2])
    for i in range(3):
        assert torch.equal(whole[:, :, i], grads[i])
    assert bool((whole[:, :, 3] == 7.0).all())
    for bad in (q, k[:, :, :], qkv[:, :, 2]):
        with pytest.raises(sk.SinkhornError):
            sk.cross_attention_grad(dout, q, k, v, out, lse, dq=bad)
    # parts that begin inside another
    inside = whole.as_strided(q.shape, q.stride(), d)
    with pytest.raises(sk.SinkhornError) as e:
        sk.cross_attention_grad(dout, q, k, v, out, lse, dq=whole[:, :, 0], dk=inside)
    assert "overlap" in str(e.value)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("Lq,Lk", [(1, 90), (1, 6000), (40, 500)])
def test_forward_in_the_callers_tensors(sk, dtype, Lq, Lk):
    (q, k, v, _), kw, extra = _case(dtype, 2, Lq, 4, 2, Lk, 64, 32, seed=47)
    mass = torch.empty(2, 2, Lk, device=DEV)
    want = sk.cross_attention(q, k, v, mass_out=mass, **kw)
    side = torch.full((2 * 4 * Lq + 64,), 7.0, device=DEV)
    weight = torch.full((2 * 2 * Lk + 64,), 7.0, device=DEV)
    out, whole = _place(want[0].shape, dtype, "behind")
    lse, got = side[32:-32].view(2, 4, Lq), weight[32:-32].view(2, 2, Lk)
    res = sk.cross_attention(q, k, v, out=out, lse=lse, mass_out=got, **kw)
    assert res[0].data_ptr() == out.data_ptr() and res[1].data_ptr() == lse.data_ptr()
    for x, y in zip((out, lse, got), (*want, mass)):
        assert torch.equal(x, y)
    assert _only(out, whole) and _only(lse, side) and _only(got, weight)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("layout", ["heads", "half", "odd", "behind"])
def test_evict_into_the_callers_tensors(sk, dtype, layout):
    """Every output given, short sequences among them: the kept places written,
    nothing beside them; and into rows of the cache's own buffer behind its keys."""
    B, n, H, d, dv, keep = 3, 700, 2, 64, 24, 130
    (_, k, v, _), kw, extra = _case(dtype, B, 1, H, H, n, d, dv, seed=48)
    lens = torch.tensor([700, 60, 131], dtype=torch.int32, device=DEV)
    want = sk.cache_evict(k, v, extra["mass"], keep, key_lengths=lens, first=3, recent=20)
    (ko, kw_), (vo, vw) = _place((B, keep, H, d), dtype, layout), _place((B, keep, H, dv), dtype, layout)
    mass, index = (torch.full((B * H * keep + 64,), 7, dtype=t, device=DEV) for t in (F32, torch.int32))
    left = torch.full((B + 64,), 7, dtype=torch.int32, device=DEV)
    views = (ko, vo, mass[32:-32].view(B, H, keep), index[32:-32].view(B, H, keep), left[32:-32])
    got = sk.cache_evict(k, v, extra["mass"], keep, key_lengths=lens, first=3, recent=20, k_out=views[0], v_out=views[1],
                         mass_out=views[2], index_out=views[3], lengths_out=views[4])
    for g, x in zip(got, views):
        assert g.data_ptr() == x.data_ptr()
    for g, w in zip(got[2:], want[2:]):
        assert torch.equal(g, w)
    for g, w in zip(got[:2], want[:2]):
        for b, c in enumerate(want[4].tolist()):
            assert torch.equal(g[b, :c], w[b, :c]) and bool((g[b, c:] == 7.0).all())
    for x, whole in zip(views, (kw_, vw, mass, index, left)):
        assert _only(x, whole)
    # one buffer for the cache and what is left of it
    both = torch.zeros(B, n + keep, H, d, dtype=dtype, device=DEV)
    both[:, :n] = k
    sk.cache_evict(both[:, :n], v, extra["mass"], keep, key_lengths=lens, first=3, recent=20, k_out=both[:, n:])
    assert torch.equal(both[:, :n], k) and torch.equal(both[:, n:], want[0])
    for at in (1, n - 1):
        with pytest.raises(sk.SinkhornError) as e:
            sk.cache_evict(both[:, :n], v, extra["mass"], keep, k_out=both[:, at:at + keep])
        assert "overlap" in str(e.value)


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "fp16"])
@pytest.mark.parametrize("B,Lq,Hq,Hkv,Lk,d,dv", [(4, 1, 8, 8, 1000, 64, 64), (2, 1, 16, 4, 5000, 128, 128), (3, 5, 12, 4, 700, 80, 96),
                                                 (1, 32, 1, 1, 333, 50, 7), (1, 1, 1, 1, 40, 32, 32)])
def test_few_rows_are_off_by_their_own_rounding(sk, dtype, B, Lq, Hq, Hkv, Lk, d, dv):
    """Where all rows fit one tile, weights enter their product in two parts,
    each rounded to u of what it holds: off by u^2 of the weight, so out is off by
    its own rounding u |out| and what fp32 leaves. (fp16: a part below the normal
    range by 2^-25, against weights that sum to 1 at least.)"""
    (q, k, v, _), ragged, _ = _case(dtype, B, Lq, Hq, Hkv, Lk, d, dv, seed=49)
    ragged["key_lengths"].clamp_(min=1)
    for kw in (dict(), dict(key_bias=ragged["key_bias"]), ragged):
        out, _ = sk.cross_attention(q, k, v, **kw)
        ref = Ref(q, k, v, **kw)
        W = (ref.P @ ref.V.abs()).permute(0, 2, 1, 3)
        weights = 1.01 * ref.u * W  # what out_tol holds for weights in one part
        assert_close(out, ref.out, ref.out_tol - weights + ref.u * weights, "out")
