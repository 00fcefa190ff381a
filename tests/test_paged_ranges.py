"""The paged cache's kernels where one warp, CTA or launch has more to do than in small cases: blocks that are
missing beside blocks that are seen in part, many segments a CTA, several heads a warp, values of any size and
references that rise; and what the calls refuse or allow of their arguments' layouts."""
import numpy as np
import pytest
import torch

import oracle
import long_context_decode_kv1b_b200 as kv
import paged_reference as ref
from test_paged import SCALE, check_attend, dev, filled, new_cache, rope_table, same_bytes, table_for

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(40)


def check_rows(out, q, cache, signs, scale, table, seen, rows, prefix=None, tolerance=ref.Row.tolerance):
    """Rows (sequence, query head) of `out` against 64 bits; sequence b sees the tokens seen(b) of its pages, and
    with prefix = (pages, tokens) those of the shared prefix first."""
    pages, got, eps = cache.pages.cpu().numpy(), ref.to_np(out).astype(np.float64), torch.finfo(q.dtype).eps
    G = q.shape[1] // cache.num_kv_heads
    for b, hq in rows:
        parts = [ref.gather(pages, table[b], hq // G, seen(b))]
        if prefix is not None:
            parts.insert(0, ref.gather(pages, prefix[0], hq // G, prefix[1]))
        row = ref.Row(ref.to_np(q[b, hq]), signs, scale, parts)
        err, tol = np.abs(got[b, hq] - row.out), tolerance(row, eps)
        assert (err <= tol).all(), f"sequence {b} head {hq}: error {err.max():.3e}, {(err / tol).max():.2f} of the tolerance"


def some_rows(rng, B, Hq, n):
    return [(int(rng.integers(B)), int(rng.integers(Hq))) for _ in range(n)] + [(0, 0), (B - 1, Hq - 1)]


# ------------------------------------------------------------------- missing blocks and blocks seen in part
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attend_missing_first_page_before_a_partial_last_block(dtype):
    # enough segments of two blocks that a warp's run holds both: the missing first block, and the last one with NaN
    # and infinities behind the length
    rng = np.random.default_rng(1)
    lengths = [int(x) for x in rng.integers(33, 64, 128)]
    cache, signs, table, _ = filled(lengths, 32, 32, 41)
    bad = table.copy()
    bad[:, 0] = -1
    q = torch.randn((128, 32, 128), device="cuda").to(dtype)
    out = cache.attend(q, SCALE, dev(bad), dev(lengths, torch.int32))
    assert cache.status() == kv.STATUS_BAD_INDEX
    assert torch.isfinite(out).all()
    check_rows(out, q, cache, signs, SCALE, table, lambda b: np.arange(32, lengths[b]), some_rows(rng, 128, 32, 60))


@pytest.mark.parametrize("window, sinks", [(40, 5), (33, 33)])
def test_attend_missing_first_tokens_before_a_window(window, sinks):
    # the page that the first kept tokens are on is missing; the block where the window begins is seen in part, and so
    # is the last one
    rng = np.random.default_rng(2)
    lengths = [int(x) for x in rng.integers(150, 220, 128)]
    cache, signs, table, _ = filled(lengths, 32, 32, 42)
    bad = table.copy()
    bad[:, (sinks - 1) // 32] = cache.num_pages
    q = (2 * torch.randn((128, 32, 128), device="cuda")).to(torch.bfloat16)
    out = cache.attend(q, SCALE, dev(bad), dev(lengths, torch.int32), window=window, sinks=sinks)
    assert cache.status() == kv.STATUS_BAD_INDEX

    def seen(b):
        t = np.arange(lengths[b])
        return t[((t >= lengths[b] - window) | (t < sinks)) & (t // 32 != (sinks - 1) // 32)]

    check_rows(out, q, cache, signs, SCALE, table, seen, some_rows(rng, 128, 32, 60))


def test_attend_shared_missing_first_page_before_a_partial_last_block():
    # the same in a short prefix that the attend's kernel takes
    rng = np.random.default_rng(3)
    lengths, prefix = [int(x) for x in rng.integers(33, 64, 16)], 57
    cache, signs, table, pre = filled(lengths, 32, 64, 43, prefix=prefix)
    missing, bad = pre.copy(), table.copy()
    missing[0] = -1
    bad[:, 0] = -1
    q = torch.randn((16, 64, 128), device="cuda", dtype=torch.float16)
    out = cache.attend_shared(q, SCALE, dev(missing), dev([prefix], torch.int32), dev(bad), dev(lengths, torch.int32))
    assert cache.status() == kv.STATUS_BAD_INDEX and torch.isfinite(out).all()
    check_rows(out, q, cache, signs, SCALE, table, lambda b: np.arange(32, lengths[b]), some_rows(rng, 16, 64, 60),
               prefix=(pre, np.arange(32, prefix)))
