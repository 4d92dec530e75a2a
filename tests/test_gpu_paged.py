"""GPU parity of attention over a paged cache against a plain form, row by row, in
64 bits (tests/paged_ref.py, which also derives the tolerances), and of the
operators around it run together."""
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


def _make(dtype, lens, m, Hq, H, d, dv, size, seed=0, gain=1.0, extra=0, layout="slots"):
    """(q, k_cache, v_cache, table, lengths) with pages in a drawn order; free pages hold NaN."""
    gen = torch.Generator().manual_seed(seed)
    pages = sum((max(n, 0) + size - 1) // size for n in lens) + 2
    table = table_of([max(n, 0) for n in lens], size, pages, gen, extra=extra)
    q = (gain * torch.randn(len(lens), m, Hq, d, generator=gen)).to(dtype).to(DEV)
    kc, vc = (torch.randn(pages, size, H, w, generator=gen).to(dtype) for w in (d, dv))
    free = torch.ones(pages, dtype=torch.bool)
    free[table[(table >= 0) & (table < pages)].long()] = False
    kc[free], vc[free] = math.nan, math.nan
    for b, n in enumerate(lens):  # and so do the places behind a sequence in its last page
        if n > 0 and n % size:
            kc[table[b, n // size], n % size:] = math.nan
            vc[table[b, n // size], n % size:] = math.inf
    if layout == "heads":
        kc, vc = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (kc, vc))
    elif layout == "both":  # keys and values of a slot side by side
        w = torch.cat([kc, vc], 3).to(DEV)
        return q, w[..., :d], w[..., d:], table.to(DEV), _ints(lens)
    return q, kc.to(DEV), vc.to(DEV), table.to(DEV), _ints(lens)


def _check(sk, args, what, out=None, lse=None, **kw):
    got, z = sk.paged_attention(*args, out=out, lse=lse, **kw)
    ref = PagedRef(*args, **kw)
    assert_close(z, ref.lse, ref.lse_tol, what + " lse")
    assert_close(got, ref.out, ref.out_tol, what + " out")
    return got, z


SHAPES = [
    # lengths, new tokens, Hq, Hkv, d, dv, page
    ([1], 1, 1, 1, 64, 64, 8),
    ([129, 7, 64], 1, 8, 2, 128, 128, 16),
    ([1000, 1, 999], 1, 4, 4, 64, 64, 32),
    ([2049], 7, 6, 2, 80, 80, 24),
    ([65, 300], 33, 2, 1, 64, 32, 16),
    ([128], 128, 4, 4, 128, 128, 64),
    ([300, 131], 130, 3, 3, 56, 64, 8),
    ([200], 200, 2, 2, 8, 8, 256),
    ([31, 40], 3, 1, 1, 32, 32, 16),
    ([96, 90], 40, 5, 1, 72, 128, 48),
    ([513], 257, 1, 1, 40, 96, 40),
    ([64], 64, 16, 1, 96, 96, 16),
    ([4000, 50], 2, 16, 1, 128, 64, 16),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_attention(sk, dtype, case):
    lens, m, Hq, H, d, dv, size = SHAPES[case]
    _log(f"paged {dtype} {SHAPES[case]}")
    args = _make(dtype, lens, m, Hq, H, d, dv, size, seed=case, extra=case % 3)
    _check(sk, args, "causal")
    _check(sk, args, "window", recent=17, first=3, scale=0.3)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("layout", ["slots", "heads", "both"])
@pytest.mark.parametrize("m", [1, 70])
def test_layouts(sk, dtype, layout, m):
    _log(f"layouts {dtype} {layout} {m}")
    args = _make(dtype, [150, 90], m, 4, 2, 64, 64, 16, seed=1, layout=layout)
    want = _check(sk, args, layout)
    # queries and outputs that are not aligned, in wider rows, and nothing beside them written
    B, _, H, d = args[0].shape
    wide = torch.full((B * m * H * (d + 3) + 1,), 7.0, dtype=dtype, device=DEV)
    q = wide[1:].view(B, m, H, d + 3)[..., :d]
    q.copy_(args[0])
    whole = torch.full((B * m * H * (d + 3) + 1,), 7.0, dtype=dtype, device=DEV)
    out = whole[1:].view(B, m, H, d + 3)[..., :d]
    before = whole.clone()
    lse = torch.empty(B, H, m, device=DEV)
    got = sk.paged_attention(q, *args[1:], out=out, lse=lse)
    assert got[0] is out and torch.equal(out, want[0]) and torch.equal(lse, want[1])
    out.fill_(7.0)
    assert torch.equal(whole, before)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("m", [4, 50])
def test_lengths(sk, dtype, m):
    """Sequences shorter than their new tokens, rows behind their queries, none at all."""
    _log(f"lengths {dtype} {m}")
    args = _make(dtype, [333, 0, 1, m - 1, m, 64], m, 4, 2, 64, 64, 16, seed=3)
    _check(sk, args, "short")
    n = _ints([m, m, 0, (m + 1) // 2, -3, 99])
    q = args[0].clone()
    for b, x in enumerate([m, m, 0, (m + 1) // 2, 0, m]):
        q[b, x:] = math.nan
    out, lse = _check(sk, (q,) + args[1:], "queries", query_lengths=n)
    assert not out[2].any() and torch.isinf(lse[2]).all()
    lens = args[4].clone()
    lens[0], lens[1] = 2 ** 31 - 1, -7  # taken as the table's places and none
    args[3][0].clamp_(0, args[1].shape[0] - 1)
    size = args[1].shape[1]
    cap = args[3].shape[1] * size
    full = lens.clone()
    full[0], full[1] = cap, 0
    a, b = sk.paged_attention(q, *args[1:4], lens, query_lengths=n), sk.paged_attention(q, *args[1:4], full, query_lengths=n)
    assert torch.equal(a[0][1:], b[0][1:]) and torch.equal(a[1][1:], b[1][1:])
    # no rows, no sequences, no places, no pages
    assert sk.paged_attention(q[:, :0], *args[1:])[0].shape == (6, 0, 4, 64)
    assert sk.paged_attention(q[:0], args[1], args[2], args[3][:0], args[4][:0])[0].shape == (0, m, 4, 64)
    for t, k, v in ((args[3][:, :0], args[1], args[2]), (args[3], args[1][:0], args[2][:0])):
        out, lse = sk.paged_attention(args[0], k, v, t, args[4])
        assert not out.any() and (lse == -math.inf).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("recent,first", [(1, 0), (1, 1), (16, 4), (63, 64), (64, 65), (100, 1000), (5000, 3), (129, 128), (1 << 70, 1 << 70)])
@pytest.mark.parametrize("m,lens", [(1, [700, 90]), (5, [700, 5]), (200, [700, 200])])
def test_windows(sk, dtype, recent, first, m, lens):
    _log(f"window {dtype} {recent} {first} {m}")
    args = _make(dtype, lens, m, 2, 1, 64, 64, 16, seed=4)
    _check(sk, args, "window", recent=recent, first=first)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("m", [1, 40])
def test_pages_behind_the_window_may_be_gone(sk, dtype, m):
    _log(f"gone {dtype} {m}")
    args = list(_make(dtype, [1000, 800], m, 4, 2, 64, 64, 8, seed=5))
    want = _check(sk, args, "all pages", recent=100, first=20)
    keep = args[3].clone()
    for b, n in enumerate([1000, 800]):
        lo = (n - m - 100 + 1) // 8  # the first page that a window reaches
        gone = args[3][b, 3:lo].clone().long()
        args[1][gone], args[2][gone] = math.nan, math.nan
        args[3][b, 3:lo] = -1
    got = sk.paged_attention(*args, recent=100, first=20)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert not torch.equal(keep, args[3])


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("m", [1, 6, 90])
@pytest.mark.parametrize("d", [64, 128])
def test_bad_pages_take_no_part(sk, dtype, m, d):
    """Pages outside the cache in the middle, at the front, all of them; far more than a wave holds."""
    _log(f"bad pages {dtype} {m} {d}")
    args = list(_make(dtype, [2600, 300, 90, 100], m, 4, 2, d, d, 8, seed=6))
    t = args[3]
    t[0, 5], t[0, 270:280], t[0, 300] = -1, args[1].shape[0], 2 ** 31 - 1
    t[1, 0] = -(2 ** 31)
    t[2, :12] = -1
    t[3, 12] = args[1].shape[0] + 5
    out, lse = _check(sk, args, "bad pages")
    assert not out[2].any() and (lse[2] == -math.inf).all()
    _check(sk, args, "bad pages, window", recent=400, first=50)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("m,lens", [(3, [70, 3]), (40, [200, 64]), (130, [257, 130])])
@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("window", [{}, {"recent": 9, "first": 2}])
def test_hidden_keys_may_hold_anything(sk, dtype, m, lens, d, window):
    """A key or value that is no number reaches the rows that see it and no other."""
    _log(f"hidden {dtype} {m} {lens} {d} {window}")
    args = _make(dtype, lens, m, 2, 2, d, d, 16, seed=7)
    out, lse = _check(sk, args, "clean", **window)
    ref = PagedRef(*args, **window)
    for what, bad in ((1, math.nan), (1, math.inf), (2, math.nan), (2, math.inf), (2, -math.inf)):
        for b, n in enumerate(lens):
            for j in {0, n - m, n - m // 2 - 1, n - 1}:
                x = args[what].clone()
                at = int(args[3][b, j // 16]), j % 16
                x[at][0, 5] = bad  # element 5 of key head 0
                a = list(args)
                a[what] = x
                o, z = sk.paged_attention(*a, **window)
                p = torch.arange(n - m, n, device=DEV)
                see = p >= j
                if window:
                    see &= (j > p - window["recent"]) | (torch.tensor(j, device=DEV) < window["first"])
                o, z = o.clone(), z.clone()
                rows = o[b, see, 0]
                if what == 2:  # a value: its column of the rows that see it, and nothing of lse
                    assert torch.equal(z, lse), (what, bad, b, j)
                    # (a weight that rounds to 0 in the element type still counts as seen in the masked
                    # tile and as 0 x bad elsewhere; neither is a number)
                    assert not torch.isfinite(rows[:, 5]).any(), (what, bad, b, j)
                    o[b, see, 0, 5] = out[b, see, 0, 5]
                elif not math.isinf(bad):
                    assert torch.isnan(rows).all() and torch.isnan(z[b, 0, see]).all(), (what, bad, b, j)
                    o[b, see, 0], z[b, 0, see] = out[b, see, 0], lse[b, 0, see]
                else:  # an infinite score either way
                    assert not torch.isfinite(z[b, 0, see]).any() or bool((args[0][b, see, 0, 5] < 0).any()), (what, bad, b, j)
                    o[b, see, 0], z[b, 0, see] = out[b, see, 0], lse[b, 0, see]
                    # rows of a wave change the reference of their weights together, so an infinite
                    # score of one may round another's weights at another place: to the tolerance,
                    # which holds for any reference
                    assert_close(o, ref.out, ref.out_tol, f"out beside an infinite score, key {j}")
                    assert_close(z, ref.lse, ref.lse_tol, f"lse beside an infinite score, key {j}")
                    continue
                assert torch.equal(o, out) and torch.equal(z, lse), (what, bad, b, j)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_rows_without_keys_that_are_no_numbers(sk, dtype):
    _log(f"rows without keys {dtype}")
    for m in (4, 60):
        args = list(_make(dtype, [m - 2, 0], m, 4, 2, 64, 64, 16, seed=8))
        want = _check(sk, args, "clean")
        q = args[0].clone()
        q[0, :2], q[1] = math.nan, math.inf
        got = sk.paged_attention(q, *args[1:])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("m", [1, 20])
def test_sharp_scores(sk, dtype, m):
    _log(f"sharp {dtype} {m}")
    args = _make(dtype, [900, 450], m, 4, 2, 64, 64, 16, seed=9, gain=12.0)
    _check(sk, args, "sharp")
    _check(sk, args, "flat", scale=1e-6)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("d,dv", [(32, 32), (64, 40), (96, 72), (128, 128)])
@pytest.mark.parametrize("m", [1, 6, 37])
@pytest.mark.parametrize("window", [{}, {"recent": 300, "first": 5}])
def test_narrow_and_wide_tables(sk, dtype, d, dv, m, window):
    # short sequences: a table with places for them alone is worked through by one workgroup
    # a row tile, one with places for many more by several
    _log(f"tables {dtype} {d} {dv} {m} {window}")
    for extra in (0, 1000):
        q, kc, vc, t, n = _make(dtype, [255, 0, 257, 512, 31, 700][:4 if m > 6 else 6], m, 4, 2, d, dv, 16, seed=d + m, extra=extra)
        _check(sk, (q, kc, vc, t, n), f"{extra} places behind", **window)
        t[3, 2], t[2, 16], t[0, 0] = -1, kc.shape[0], 1 << 30
        _check(sk, (q, kc, vc, t, n), f"bad pages, {extra} places behind", **window)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("d", [64, 128])
def test_long_sequences_split(sk, dtype, d):
    """Many tiles a workgroup and many splits, page numbers beyond what a wave holds at a time."""
    _log(f"long {dtype} {d}")
    args = _make(dtype, [9000, 33, 5000], 1, 4, 2, d, d, 8, seed=10)
    _check(sk, args, "long")
    _check(sk, args, "long window", recent=4444, first=40)
    args = _make(dtype, [7000], 24, 4, 1, d, d, 8, seed=11)
    _check(sk, args, "chunk")


@pytest.mark.parametrize("B,H", [(9, 1), (3, 5), (70, 1)])
@pytest.mark.parametrize("m", [1, 36])
def test_numbers_of_heads(sk, B, H, m):
    _log(f"heads {B} {H} {m}")
    lens = [m + (37 * b) % 150 for b in range(B)]
    _check(sk, _make(BF, lens, m, H, H, 32, 32, 16, seed=12), "heads")


@pytest.mark.parametrize("Hq,m", [(48, 20), (96, 3), (33, 11), (40, 1), (64, 1), (5, 60)])
def test_groups_across_tiles(sk, Hq, m):
    _log(f"groups {Hq} {m}")
    _check(sk, _make(HF, [100, 77], m, Hq, 1, 64, 64, 8, seed=13), "groups")


def test_shared_pages_and_table_views(sk):
    """Two sequences with the same first pages, and a table that is a view of a wider one."""
    _log("shared pages")
    args = list(_make(BF, [200, 260], 3, 4, 2, 64, 64, 16, seed=14))
    args[3][1, :8] = args[3][0, :8]
    wide = torch.full((2, 40), -1, dtype=torch.int32, device=DEV)
    wide[:, :args[3].shape[1]] = args[3]
    args[3] = wide[:, :args[3].shape[1]]
    a = _check(sk, args, "shared")
    args[3] = wide
    b = _check(sk, args, "wider")
    assert torch.equal(a[1][:, :, :1].isfinite(), b[1][:, :, :1].isfinite())


def test_caches_beyond_32_bits(sk):
    """Pages whose elements lie beyond 2^32, and heads more than 4 GB apart."""
    _log("large cache")
    size, H, d, pages = 64, 8, 128, 72000
    kc = torch.empty(pages, size, H, d, dtype=BF, device=DEV)
    vc = torch.empty(pages, size, H, d, dtype=BF, device=DEV)
    for m in (1, 50):
        small = _make(BF, [250, 300], m, 16, H, d, d, size, seed=15)
        ids = _ints([71999, 3, 71998, 36000, 65536, 70000, 1, 40000, 0, 71000, 2])[:small[1].shape[0]]
        kc[ids.long()], vc[ids.long()] = small[1], small[2]
        t = small[3].clone()
        ok = (t >= 0) & (t < small[1].shape[0])
        t[ok] = ids[t[ok].long()]
        want = sk.paged_attention(*small)
        got = sk.paged_attention(small[0], kc, vc, t, small[4])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # [heads, pages, slots, width], a head 4.5 GB
    kh = torch.empty(2, 275000, size, d, dtype=BF, device=DEV).permute(1, 2, 0, 3)
    small = _make(BF, [250, 300], 5, 4, 2, d, d, size, seed=16)
    ids = _ints([274999, 3, 1, 0, 9, 7, 70000, 270000, 5, 11, 2])[:small[1].shape[0]]
    kh[ids.long()] = small[1]
    vh = torch.empty(2, 275000, size, d, dtype=BF, device=DEV).permute(1, 2, 0, 3)
    vh[ids.long()] = small[2]
    t = small[3].clone()
    ok = (t >= 0) & (t < small[1].shape[0])
    t[ok] = ids[t[ok].long()]
    want, got = sk.paged_attention(*small), sk.paged_attention(small[0], kh, vh, t, small[4])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("m", [1, 70])
@pytest.mark.parametrize("back", [0, 3, 100])
def test_sequences_that_end_next_to_2_31(sk, dtype, m, back):
    """One page of 2^31 - 8 slots that all lie in the same place: out is the value, lse the
    score plus the log of the visible keys' number."""
    _log(f"2^31 {dtype} {m} {back}")
    size, d = 2 ** 31 - 8, 64
    n = size - back
    k = torch.full((1, 1, 1, d), 0.25, dtype=dtype, device=DEV).expand(1, size, 1, d)
    v = torch.linspace(-8, 8, 64, device=DEV).round().to(dtype).view(1, 1, 1, d).expand(1, size, 1, d)
    q = torch.full((1, m, 2, d), 0.5, dtype=dtype, device=DEV)
    for kw in ({"recent": 100}, {"recent": 100, "first": 7}, {"recent": 2 ** 31 - 200}, {}):
        out, lse = sk.paged_attention(q, k, v, _ints([[0]]), _ints([n]), scale=0.125, **kw)
        p = n - m + torch.arange(m, dtype=torch.float64)  # places
        recent = float(kw.get("recent", 2 ** 31))
        seen = torch.minimum(p + 1, torch.full_like(p, recent + kw.get("first", 0)))
        want = (1.0 + seen.log()).view(1, 1, m).expand(1, 2, m)
        # scores are 1; weights 1 and their sums, whole numbers, are rounded to 24 bits
        # when lanes and splits are joined, ten times at most; then a logarithm and a sum
        assert_close(lse, want, torch.full_like(want, 2.0 ** -24 * (10 + 8 * 32)), f"lse {kw}")
        # split 512 times a lane's sums are whole numbers below 2^24 times the value, exact; the
        # bound leaves room for splits 2^11 times longer, then the joins' roundings and the result's
        tol = (v[0, 0, 0].double().abs() * (2.0 ** -13 + (2.0 ** -8 if dtype == BF else 0.0)) + 2.0 ** -40).cpu()
        assert_close(out, v[0, 0, 0].double().cpu().expand(1, m, 2, d), tol.expand(1, m, 2, d), f"out {kw}")


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_as_cross_attention(sk, dtype):
    """A last token that sees all keys: the contiguous operator's results, to both tolerances."""
    _log(f"as cross attention {dtype}")
    B, n, Hq, H, d, size = 2, 500, 4, 2, 64, 16
    args = _make(dtype, [n, n], 1, Hq, H, d, d, size, seed=17)
    need = (n + size - 1) // size
    k, v = (c[args[3][:, :need].long()].reshape(B, -1, H, d)[:, :n].contiguous() for c in args[1:3])
    out, lse = sk.cross_attention(args[0], k, v)
    ref = PagedRef(*args)
    assert_close(out, ref.out, ref.out_tol, "contiguous out")
    assert_close(lse, ref.lse, ref.lse_tol, "contiguous lse")
    _check(sk, args, "paged")


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("window", [{}, {"recent": 20, "first": 4}])
def test_prompt_then_tokens(sk, dtype, window):
    """The operators together: a ragged batch of prompts is appended and attended to in chunks,
    then tokens follow one by one; every row is as if its whole sequence had been taken at once."""
    _log(f"together {dtype} {window}")
    B, Hq, H, d, size, P, N = 3, 4, 2, 64, 16, 50, 12
    gen = torch.Generator().manual_seed(18)
    prompt, chunk = [50, 1, 33], 20
    lens = [p + N for p in prompt]
    pages = sum((n + size - 1) // size for n in lens) + 1
    table = table_of(lens, size, pages, gen).to(DEV)
    total = P + N
    x = [torch.randn(B, total, h, d, generator=gen).to(dtype).to(DEV) for h in (Hq, H, H)]
    w = [(1 + 0.2 * torch.randn(d, generator=gen)).to(DEV) for _ in range(2)]
    kw = dict(frequencies=sk.rotary_frequencies(d, device=DEV), norm_eps=1e-6)
    kc, vc = (torch.full((pages, size, H, d), math.nan, dtype=dtype, device=DEV) for _ in range(2))
    have = _ints([0] * B)
    outs = [[] for _ in range(B)]
    start = 0
    while start < P:  # chunks of the prompts
        n = [min(max(p - start, 0), chunk) for p in prompt]
        sl = slice(start, start + chunk)
        have, q = sk.cache_append(x[1][:, sl], x[2][:, sl], kc, vc, table, have, new_lengths=_ints(n)[:], q=x[0][:, sl],
                                  q_weight=w[0], k_weight=w[1], **kw)
        out, _ = sk.paged_attention(q, kc, vc, table, have, query_lengths=_ints(n), **window)
        for b in range(B):
            outs[b].append(out[b, :n[b]])
        start += chunk
    for t in range(N):  # then one token each, placed behind its own prompt
        at = [p + t for p in prompt]
        tok = [torch.stack([y[b, at[b]] for b in range(B)])[:, None] for y in x]
        have, q = sk.cache_append(tok[1], tok[2], kc, vc, table, have, q=tok[0], q_weight=w[0], k_weight=w[1], **kw)
        out, _ = sk.paged_attention(q, kc, vc, table, have, **window)
        for b in range(B):
            outs[b].append(out[b])
    assert have.tolist() == lens
    # the whole sequences at once: rotated contiguously, then put into pages by a plain append
    qr, kr = sk.rotate_heads(x[0], x[1], q_weight=w[0], k_weight=w[1], **kw)
    k2, v2 = (torch.zeros_like(kc) for _ in range(2))
    have2, _ = sk.cache_append(kr, x[2], k2, v2, table, _ints([0] * B), new_lengths=_ints(lens))
    for b in range(B):
        ids = table[b, :(lens[b] + size - 1) // size].long()
        for a, c in ((kc, k2), (vc, v2)):
            assert torch.equal(a[ids].flatten(0, 1)[:lens[b]], c[ids].flatten(0, 1)[:lens[b]])
        ref = PagedRef(qr[b:b + 1, :lens[b]], k2, v2, table[b:b + 1], _ints([lens[b]]), **window)
        got = torch.cat(outs[b])[None]
        # few rows hold the weights in two parts, many in one: the wider tolerance covers both
        assert_close(got, ref.out, ref.out_tol, f"sequence {b}")


def test_streams_graphs_and_repeats(sk):
    """Two captured steps with workspaces of their own, replayed side by side while lengths change."""
    _log("graphs")
    gen = torch.Generator().manual_seed(19)
    a = list(_make(BF, [3000, 2500], 1, 8, 2, 128, 128, 16, seed=20))
    c = list(_make(BF, [900, 1000], 40, 8, 2, 128, 128, 16, seed=21))
    want = [sk.paged_attention(*x) for x in (a, c)]
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(sk.paged_attention(*a), want[0]))
    graphs, res, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for x in (a, c):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res.append(sk.paged_attention(*x))
        graphs.append(g)
    for n in range(3):
        lens = [torch.randint(200, 2500, (2,), generator=gen).int(), torch.randint(40, 900, (2,), generator=gen).int()]
        for x, y in zip((a, c), lens):
            x[4].copy_(y)
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for x, r in zip((a, c), res):
            for y, z in zip(sk.paged_attention(*x), r):
                assert torch.equal(y, z)
