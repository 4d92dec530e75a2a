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
