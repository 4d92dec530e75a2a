"""GPU parity of appending to a paged cache against a plain form, token by
token, in 64 bits (tests/paged_ref.py, which also derives the tolerances)."""
import math
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from attention_ref import assert_close  # noqa: E402
from paged_ref import append_ref, table_of  # noqa: E402

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


def _cache(gen, pages, size, H, d, dtype, layout):
    """[pages, size, H, d] in several layouts of memory, filled with numbers."""
    t = torch.randn(pages, size, H, d, generator=gen).to(dtype).to(DEV)
    if layout == "slots":
        return t
    if layout == "heads":  # [pages, H, size, d]
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    if layout == "odd":
        w = torch.full((t.numel() // d * (d + 3) + 1,), 7.0, dtype=dtype, device=DEV)
        x = w[1:].view(pages, size, H, d + 3)[..., :d]
        x.copy_(t)
        return x
    raise ValueError(layout)


def _check(sk, what, k, v, k_cache, v_cache, table, before, **kw):
    want = append_ref(k, v, k_cache, v_cache, table, before, **kw)
    lens, q = sk.cache_append(k, v, k_cache, v_cache, table, before, **kw)
    assert_close(k_cache, want[0], want[1], what + " keys")
    assert_close(v_cache, want[2], torch.zeros(()), what + " values")
    assert torch.equal(lens.cpu(), want[3]), what
    if kw.get("q") is not None:
        assert_close(q, want[4], want[5], what + " queries")
    else:
        assert q is None
    return lens, q


CASES = [
    # new tokens, cached, Hq, Hkv, d, dv, rotated, page
    ([1, 1, 1, 1], [0, 7, 8, 100], 4, 2, 64, 64, 64, 8),
    ([1, 1], [31, 4095], 8, 8, 128, 128, 128, 16),
    ([5, 17, 0, 40], [0, 3, 9, 23], 3, 1, 80, 80, 40, 24),
    ([300, 1], [0, 255], 2, 2, 64, 128, 32, 256),
    ([33, 20], [5, 48], 0, 4, 72, 8, 72, 16),
    ([9, 9, 9], [0, 0, 1], 4, 4, 50, 33, 26, 40),
    ([130], [1], 6, 2, 96, 64, 0, 64),
    ([3, 2], [10, 11], 1, 1, 1, 1, 0, 8),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "pairs"])
@pytest.mark.parametrize("layout", ["slots", "heads", "odd"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_append(sk, dtype, interleaved, layout, case):
    new, old, Hq, H, d, dv, r, size = CASES[case]
    _log(f"append {dtype} {interleaved} {layout} {CASES[case]}")
    gen = torch.Generator().manual_seed(case)
    B, L = len(new), max(new)
    lens = [a + b for a, b in zip(new, old)]
    pages = sum((n + size - 1) // size for n in lens) + 2
    table = table_of(lens, size, pages, gen, extra=case % 3).to(DEV)
    mk = lambda H, w: torch.randn(B, L, H, w, generator=gen).to(dtype).to(DEV)  # noqa: E731
    proj = mk(Hq + H, d)  # queries and keys side by side
    q, k, v = (proj[:, :, :Hq] if Hq else None), proj[:, :, Hq:], mk(H, dv)
    kc, vc = _cache(gen, pages, size, H, d, dtype, layout), _cache(gen, pages, size, H, dv, dtype, layout)
    common = dict(new_lengths=_ints(new), q=q, frequencies=sk.rotary_frequencies(r, device=DEV) if r else None,
                  interleaved=interleaved, gain=1.1)
    _check(sk, "rotated", k, v, kc, vc, table, _ints(old), **common)
    w = [(1 + 0.2 * torch.randn(d, generator=gen)).to(DEV) for _ in range(2)]
    _check(sk, "normed", k, v, kc, vc, table, _ints(old), norm_eps=1e-6, k_weight=w[0], q_weight=w[1] if Hq else None, **common)
    if r:
        pos = torch.randint(0, 1 << 20, (B, L), generator=gen).int().to(DEV)
        _check(sk, "positions", k, v, kc, vc, table, _ints(old), positions=pos, **common)
    _check(sk, "as they are", k, v, kc, vc, table, _ints(old), new_lengths=_ints(new))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_bad_pages_and_full_tables(sk, dtype):
    """Places without a page, behind the table or before it are not written; nothing else is."""
    _log(f"bad pages {dtype}")
    gen = torch.Generator().manual_seed(5)
    size, H, d, B, L = 8, 2, 64, 6, 12
    table = torch.tensor([[0, -1, 1], [2, 12, 3], [4, 5, 2 ** 31 - 1], [6, 7, 8], [9, -(2 ** 31), 10], [11, 11, 11]],
                         dtype=torch.int32, device=DEV)
    table[5] = _ints([11, -1, -1])
    before = _ints([4, 4, 16, 20, -5, 2 ** 31 - 1])
    k = torch.randn(B, L, H, d, generator=gen).to(dtype).to(DEV)
    v = torch.randn(B, L, H, d, generator=gen).to(dtype).to(DEV)
    kc, vc = (_cache(gen, 12, size, H, d, dtype, "slots") for _ in range(2))
    f = sk.rotary_frequencies(d, device=DEV)
    lens, _ = _check(sk, "bad pages", k, v, kc, vc, table, before, frequencies=f)
    assert lens.tolist() == [16, 16, 24, 24, 12, 24]
    _check(sk, "lengths", k, v, kc, vc, table, before, frequencies=f, new_lengths=_ints([-1, 99, 3, 0, 12, 1]))
    # no places, no pages, no tokens, no sequences
    for t, c in ((table[:, :0], kc), (table, kc[:0])):
        cc, vv = c, vc[:c.shape[0]]
        old = cc.clone()
        lens, _ = sk.cache_append(k, v, cc, vv, t, before)
        cap = t.shape[1] * size
        assert lens.tolist() == [min(max(int(n), 0), cap) + min(L, cap - min(max(int(n), 0), cap)) for n in before]
        assert torch.equal(cc, old)
    none = k[:, :0]
    lens, q = sk.cache_append(none, none, kc, vc, table, before, q=none, frequencies=f)
    assert lens.tolist() == [4, 4, 16, 20, 0, 24] and q.shape == none.shape
    lens, _ = sk.cache_append(k[:0], v[:0], kc, vc, table[:0], before[:0])
    assert lens.shape == (0,)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_rows_that_are_no_numbers(sk, dtype):
    """Padding holds anything; a token that is no number spoils its own place alone."""
    _log(f"no numbers {dtype}")
    gen = torch.Generator().manual_seed(6)
    size, H, d, B, L = 16, 2, 64, 2, 6
    table = table_of([40, 40], size, 8, gen).to(DEV)
    k, v, q = (torch.randn(B, L, H, d, generator=gen).to(dtype).to(DEV) for _ in range(3))
    kw = dict(new_lengths=_ints([6, 2]), frequencies=sk.rotary_frequencies(d, device=DEV), norm_eps=1e-6)
    before = _ints([13, 30])
    a = [_cache(gen, 8, size, H, d, dtype, "slots") for _ in range(2)]
    b = [x.clone() for x in a]
    qa = sk.cache_append(k, v, *a, table, before, q=q, **kw)[1]
    for t in (k, v, q):
        t[1, 2:] = math.nan
        t[0, 3, 1] = math.inf
    qb = sk.cache_append(k, v, *b, table, before, q=q, **kw)[1]
    page, slot = int(table[0, 1]), 0  # place 16 of sequence 0
    for x, y in zip(a, b):
        assert not torch.isfinite(y[page, slot, 1].float()).all()
        y[page, slot, 1] = x[page, slot, 1]
        assert torch.equal(x, y)
    qb[0, 3, 1] = qa[0, 3, 1]
    assert torch.equal(qa, qb)


def test_places_beyond_32_bits(sk):
    """A cache of 9 GB a side: pages whose elements lie beyond 2^32."""
    _log("large cache")
    gen = torch.Generator().manual_seed(7)
    size, H, d, pages = 64, 8, 128, 72000
    assert pages * size * H * d > 2 ** 32
    kc = torch.empty(pages, size, H, d, dtype=BF, device=DEV)
    vc = torch.empty(pages, size, H, d, dtype=BF, device=DEV)
    ids = [71999, 3, 71998, 36000, 65536]
    table = _ints([ids])
    k, v = (torch.randn(1, 300, H, d, generator=gen).to(BF).to(DEV) for _ in range(2))
    f = sk.rotary_frequencies(d, device=DEV)
    small = [torch.zeros(5, size, H, d, dtype=BF, device=DEV) for _ in range(2)]
    sk.cache_append(k, v, *small, _ints([[0, 1, 2, 3, 4]]), _ints([20]), frequencies=f)
    for c in (kc, vc):
        c[ids] = 0
    sk.cache_append(k, v, kc, vc, table, _ints([20]), frequencies=f)
    assert torch.equal(kc[ids], small[0]) and torch.equal(vc[ids], small[1])
    # the same by strides of one buffer that holds keys and values of a page side by side
    both = torch.zeros(5, 2, size, H, d, dtype=BF, device=DEV)
    sk.cache_append(k, v, both[:, 0], both[:, 1], _ints([[0, 1, 2, 3, 4]]), _ints([20]), frequencies=f)
    assert torch.equal(both[:, 0], small[0]) and torch.equal(both[:, 1], small[1])


def test_graph_of_a_growing_cache(sk):
    """Captured steps that append at device lengths, replayed as the cache grows, with eager work between."""
    _log("graph")
    gen = torch.Generator().manual_seed(8)
    size, H, d, B, steps = 8, 2, 64, 3, 20
    table = table_of([steps + 5] * B, size, 16, gen).to(DEV)
    k, v, q = (torch.empty(B, 1, H, d, dtype=BF, device=DEV) for _ in range(3))
    lens = _ints([0, 5, 3])
    f = sk.rotary_frequencies(d, device=DEV)
    a = [torch.zeros(16, size, H, d, dtype=BF, device=DEV) for _ in range(2)]
    b = [x.clone() for x in a]
    kw = dict(frequencies=f, norm_eps=1e-6)
    sk.cache_append(k.zero_(), v.zero_(), *a, table, lens, q=q.zero_(), **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, qo = sk.cache_append(k, v, *a, table, lens, q=q, **kw)
        lens.copy_(out)
    lens.copy_(_ints([0, 5, 3]))
    for x in a:
        x.zero_()
    eager = _ints([0, 5, 3])
    for _ in range(steps):
        new = torch.randn(3, B, 1, H, d, generator=gen).to(BF).to(DEV)
        k.copy_(new[0])
        v.copy_(new[1])
        q.copy_(new[2])
        graph.replay()
        eager, qe = sk.cache_append(new[0], new[1], *b, table, eager, q=new[2], **kw)
        torch.cuda.synchronize()
        assert torch.equal(lens, eager) and torch.equal(qo, qe)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_lengths_next_to_2_31(sk):
    """The new length stays within the table where the sum would pass 2^31 (no page: nothing is written)."""
    _log("lengths next to 2^31")
    size = 2 ** 31 - 8
    kc = torch.empty(0, size, 1, 8, dtype=BF, device=DEV)
    k = torch.ones(3, 20, 1, 8, dtype=BF, device=DEV)
    lens, _ = sk.cache_append(k, k, kc, kc.clone(), _ints([[0], [0], [0]]), _ints([size - 5, 2 ** 31 - 1, size - 30]))
    assert lens.tolist() == [size, size, size - 10]


def test_calls_beyond_the_last_cache(sk):
    """More than 256 MB in a call (written past the caches) as in parts: the same bits."""
    _log("beyond the cache")
    B, L, H, d, size = 4, 6000, 16, 128, 32
    gen = torch.Generator(device=DEV).manual_seed(4)
    k, v, q = (torch.randn(B, L, h, d, generator=gen, device=DEV).to(BF) for h in (H, H, 8))
    assert 4 * k.numel() * 2 > 1 << 28 > 4 * (2 * k[0].numel() + q[0].numel())
    pages = B * (L // size + 1)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(5)).to(torch.int32).view(B, -1).to(DEV)
    before = _ints([0, 5, 31, 32])
    a, b = (torch.zeros(2, pages, size, H, d, dtype=BF, device=DEV) for _ in range(2))
    kw = dict(frequencies=sk.rotary_frequencies(d, device=DEV))
    lens, out = sk.cache_append(k, v, a[0], a[1], table, before, q=q, **kw)
    for i in range(B):
        n, o = sk.cache_append(k[i:i + 1], v[i:i + 1], b[0], b[1], table[i:i + 1], before[i:i + 1], q=q[i:i + 1], **kw)
        assert torch.equal(n, lens[i:i + 1]) and torch.equal(o, out[i:i + 1])
    assert torch.equal(a, b)
