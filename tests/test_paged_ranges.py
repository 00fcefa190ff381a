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


# ------------------------------------------------------------------------------------- values of every size
def unit_tolerance(row, eps):
    """As Row.tolerance, but what small weights may lose goes with the values' size: a block's scales enter the products
    as their multiple of a power of two whose largest is below 2 and at least 2^-7 where they are ordinary (unit 1),
    else at least 2^-3 (unit at most 8 of the largest scale).  A token's weight scale may lose 2^-25 of the unit, 2^4 more
    where its code sits four bits higher, times a code of 15, behind a reference of 2^7: 2^-24 of the unit.  Its weight
    as a subnormal loses 2^-25, 2^-21 where it is lowered, behind 2^7: 2^-32 of the largest |value|, twice for the
    normaliser, and 2^-28 of 15 scales.  Scales of 2 or more come down by their power of two and may lose 2^-25 of
    15 units each time their weight counts.  Minima that are subnormal operands: a product of theirs keeps 2^-38 of
    its largest weight, 17 terms."""
    if row.tokens == 0:
        return np.full(ref.D, 1e-30)
    unit = 8 * row.step if row.step < 2.0 ** -7 else max(1.0, 8 * row.step if row.step >= 2 else 1.0)
    rel = 3 * 2.0 ** -11 + 2 * (16 * 2.0 ** -24 * row.mag + 2.0 ** -21) + 2.0 ** -18
    tail = row.tokens * (2.0 ** -24 * unit + 2.0 ** -31 * row.largest + 2.0 ** -24 * row.step)
    tail += 2.0 ** -21 * unit * (row.step >= 2) + 17 * 2.0 ** -38
    part = 2.0 ** -11 if eps > 2.0 ** -9 else 2.0 ** -13
    return (1 + eps) * (rel * row.spread + part * row.reach + tail) + eps / 2 * np.abs(row.out) + 2.0 ** -25


def sized_cache(n, H, size, lead, growing=False, page=64):
    """A cache of one list of pages with n tokens of normal values of a size (growing: from a 1024th of it on), the logits
    of one token `lead` above the others' for queries near `q`; (cache, signs, pages, q of a kv-head)."""
    g = torch.Generator(device="cuda").manual_seed(46)
    num = (n + page - 1) // page
    cache, signs = new_cache(num + 1, H, page)
    k, v = torch.randn((2, n, H, 128), generator=g, device="cuda")
    q = torch.randn((H, 128), generator=g, device="cuda")
    k *= 0.05
    # the 1-bit key of 0.05 z + a q reads q at about its norm: logit |q|^2 a / sqrt(128) over the others'
    k[n // 3] = q * (lead / (q.square().sum(1, keepdim=True) * SCALE))
    v *= size
    if growing:
        v *= torch.logspace(-10, 0, n, base=2.0, device="cuda")[:, None, None]
    v.clamp_(-65504, 65504)
    pages = np.random.default_rng(46).permutation(num).astype(np.int32)
    cache.append(k, v, dev(pages[None]), dev([0], torch.int32), dev([0, n], torch.int32))
    return cache, signs, pages, q


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n, lead", [(860, 8.0), (4096, 0.0), (4096, 6.0)])
@pytest.mark.parametrize("size", [3e-6, 1e-5, 1e-4, 1e-3, 0.03, 1.0, 40.0, 30000.0])
def test_attend_values_of_every_size(size, n, lead, dtype):
    # one run of tokens a warp, so that the leading token is the reference of the others: 148 x 12 segments at least
    H, G = 2, 4
    cache, signs, pages, q1 = sized_cache(n, H, size, lead)
    B = 148 * 12 // H // 2
    q = (q1[:, None].expand(H, G, 128).reshape(1, H * G, 128) + 0.02 * torch.randn((B, H * G, 128), device="cuda")).to(dtype)
    table = np.tile(pages, (B, 1))
    out = cache.attend(q, SCALE, dev(table), dev([n] * B, torch.int32))
    assert cache.status() & ~kv.STATUS_FP16_SATURATED == 0
    rows = some_rows(np.random.default_rng(6), B, H * G, 12)
    check_rows(out, q, cache, signs, SCALE, table, lambda b: np.arange(n), rows, tolerance=unit_tolerance)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("size", [1e-2, 8.0, 60000.0])
def test_attend_values_that_grow_or_fall(size, turned, dtype):
    # sizes that change by 2^10 along a warp's run, up or down, with a flat softmax
    n, H, G = 1500, 2, 2
    cache, signs, pages, q1 = sized_cache(n, H, size, 0.0, growing=True)
    if turned:  # whole pages back to front
        n = n // 64 * 64
        pages = pages[:n // 64][::-1].copy()
    B = 500
    q = (q1[:, None].expand(H, G, 128).reshape(1, H * G, 128) + torch.randn((B, H * G, 128), device="cuda")).to(dtype)
    table = np.tile(pages, (B, 1))
    out = cache.attend(q, SCALE, dev(table), dev([n] * B, torch.int32))
    rows = some_rows(np.random.default_rng(7), B, H * G, 12)
    check_rows(out, q, cache, signs, SCALE, table, lambda b: np.arange(n), rows, tolerance=unit_tolerance)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("growing", [False, True])
@pytest.mark.parametrize("rows", [32, 160])
@pytest.mark.parametrize("size", [1e-5, 1e-3, 40.0, 60000.0])
def test_matrix_prefix_values_of_every_size(size, rows, growing, dtype):
    # a prefix that the matrix kernel takes, values small, large or growing along it, one token ahead
    n, H, G = 9000, 8, 4
    cache, signs, pages, q1 = sized_cache(n, H, size, 5.0, growing=growing)
    B = rows // G
    q = (q1[:, None].expand(H, G, 128).reshape(1, H * G, 128) + 0.1 * torch.randn((B, H * G, 128), device="cuda")).to(dtype)
    wide = np.full((40000 // 64,), -1, np.int32)
    wide[:len(pages)] = pages
    own = np.tile(pages[5:6], (B, 1))  # and own tokens of the same sizes
    lengths = [int(x) for x in np.arange(B) % 60]
    out = cache.attend_shared(q, SCALE, dev(wide), dev([n], torch.int32), dev(own), dev(lengths, torch.int32))
    assert cache.status() & ~kv.STATUS_FP16_SATURATED == 0
    check_rows(out, q, cache, signs, SCALE, own, lambda b: np.arange(lengths[b]), some_rows(np.random.default_rng(8), B, H * G, 6),
               prefix=(pages, np.arange(n)), tolerance=unit_tolerance)


# ------------------------------------------------------------------- references that rise in the matrix kernel
def rising(kind, n):
    """Factors of the query along the tokens: its share of each key, so logits of about 11 times it."""
    x = np.linspace(0, 1, n)
    return {"rising": 8 * x, "falling": 8 - 8 * x, "steps": np.floor(6 * x) * 1.3, "late": np.where(x > 0.9, 5.0, 0.1),
            "low first": np.where(np.arange(n) % 1200 < 64, 0.0, 0.35)}[kind]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows", [32, 132, 160])
@pytest.mark.parametrize("kind", ["rising", "falling", "steps", "late", "low first"])
def test_matrix_prefix_references_that_rise(kind, rows, dtype):
    # every row, a few rows of a warp or none have logits that pass what the first tokens set
    n, H, G, page = 20000, 8, 4, 64
    g = torch.Generator(device="cuda").manual_seed(47)
    num = (n + page - 1) // page
    cache, signs = new_cache(num + 1, H, page)
    k = 0.3 * torch.randn((n, H, 128), generator=g, device="cuda")
    v = torch.randn((n, H, 128), generator=g, device="cuda")
    q1 = torch.randn((H, 128), generator=g, device="cuda")
    k += dev(rising(kind, n), torch.float32)[:, None, None] * q1
    B = rows // G
    share = torch.ones((B, 1, G, 1), device="cuda")
    if B % 2 == 0:
        share[1::3] = 0.1      # rows that hardly rise among those that do
        share[2::5] = -1.0     # and rows whose logits fall
    q = (share * q1[None, :, None] + 0.1 * torch.randn((B, H, G, 128), generator=g, device="cuda")).reshape(B, H * G, 128).to(dtype)
    pages = np.random.default_rng(47).permutation(num).astype(np.int32)
    cache.append(k, v, dev(pages[None]), dev([0], torch.int32), dev([0, n], torch.int32))
    wide = np.full((40000 // page,), -1, np.int32)
    wide[:num] = pages
    own = np.tile(pages[:1], (B, 1))
    lengths = [int(x) for x in np.arange(B) % 50]
    args = (q, SCALE, dev(wide), dev([n], torch.int32), dev(own), dev(lengths, torch.int32))
    out = cache.attend_shared(*args)
    assert cache.status() == 0 and torch.equal(out, cache.attend_shared(*args))
    picks = some_rows(np.random.default_rng(9), B, H * G, 6) + [(1, 3), (2, 3)]
    check_rows(out, q, cache, signs, SCALE, own, lambda b: np.arange(lengths[b]), picks, prefix=(pages, np.arange(n)))


def test_matrix_prefix_low_first_tokens_take_no_longer():
    # 64 first tokens that score low, then all higher than them by some 2^5: the reference rises once, where rows that
    # kept the first one sent their warps through each job three times (1.8 times as long).  148 heads: one token range
    n, H, G, B, page = 4096, 148, 4, 33, 128
    g = torch.Generator(device="cuda").manual_seed(48)
    q1 = torch.randn((H, 128), generator=g, device="cuda")
    q = (q1[None, :, None] + 0.1 * torch.randn((B, H, G, 128), generator=g, device="cuda")).reshape(B, H * G, 128).to(torch.bfloat16)
    share = torch.full((n, 1, 1), 0.3, device="cuda")
    calls = []
    for low in (False, True):
        cache, _ = new_cache(n // page, H, page)
        if low:
            share[:64] = 0.0
        k = (0.3 * torch.randn((n, H, 128), generator=g, device="cuda") + share * q1).to(torch.bfloat16)
        pages = torch.arange(n // page, dtype=torch.int32, device="cuda")
        cache.append(k, k, pages[None], dev([0], torch.int32), dev([0, n], torch.int32))
        calls.append(lambda c=cache, args=(q, SCALE, pages, dev([n], torch.int32), pages[:1].repeat(B)[:, None],
                                           dev([0] * B, torch.int32)): c.attend_shared(*args))
    best = [1e9, 1e9]
    for _ in range(6):
        for i, call in enumerate(calls):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            torch.cuda.synchronize()
            a.record()
            for _ in range(10):
                call()
            b.record()
            torch.cuda.synchronize()
            best[i] = min(best[i], a.elapsed_time(b))
    assert best[1] < 1.5 * best[0], best


# --------------------------------------------------------------------- more segments than a CTA takes at once
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("heads, group", [(8, 8), (16, 2)])
def test_attend_more_segments_than_a_round(heads, group, dtype):
    # 1,024 sequences x heads over 148 CTAs: more than the 256 / group, at most 64, segments that a CTA holds
    rng = np.random.default_rng(4)
    lengths = [int(x) for x in rng.integers(0, 71, 1024)]
    lengths[5] = lengths[1023] = 0
    lengths[700] = 900
    cache, signs, table, _ = filled(lengths, 32, heads, 44)
    q = (2 * torch.randn((1024, heads * group, 128), device="cuda")).to(dtype)
    args = (q, SCALE, dev(table), dev(lengths, torch.int32))
    out = cache.attend(*args)
    assert cache.status() == 0 and torch.equal(out, cache.attend(*args))
    assert (out[5] == 0).all() and (out[1023] == 0).all()
    rows = some_rows(rng, 1024, heads * group, 300) + [(700, h) for h in range(heads * group)]
    check_rows(out, q, cache, signs, SCALE, table, lambda b: np.arange(lengths[b]), rows)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("group", [4, 8])
def test_attend_shared_more_own_segments_than_a_round(group, dtype):
    # 2,048 segments of one block on the 20 CTAs that the prefix's token ranges leave to them
    rng = np.random.default_rng(5)
    lengths, prefix = [int(x) for x in rng.integers(0, 33, 256)], 30000
    lengths[9] = 0
    cache, signs, table, pre = filled(lengths, 32, 8, 45, prefix=prefix, width=1)
    q = (2 * torch.randn((256, 8 * group, 128), device="cuda")).to(dtype)
    args = (q, SCALE, dev(pre), dev([prefix], torch.int32), dev(table), dev(lengths, torch.int32))
    out = cache.attend_shared(*args)
    assert cache.status() == 0 and torch.equal(out, cache.attend_shared(*args))
    check_rows(out, q, cache, signs, SCALE, table, lambda b: np.arange(lengths[b]), some_rows(rng, 256, 8 * group, 40) + [(9, 3)],
               prefix=(pre, np.arange(prefix)))


# ----------------------------------------------------------------------- the prompt encoder with several heads a warp
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("heads, tokens, q_heads, rot, sections, interleaved", [
    (32, 2200, 40, 128, [64], False),             # two heads a warp, query rows in two parts a token
    (33, 4500, 33, 64, [32], True),               # four and a last one
    (3, 51000, 3, 128, [16, 24, 24], False),      # four, of which there are three
    (10, 10500, 80, 80, [40], False),             # three, a last one; rotary widths that are read again
    (8, 16600, 8, 0, [], False),
])
def test_append_of_several_heads_a_warp(heads, tokens, q_heads, rot, sections, interleaved, dtype):
    # byte for byte what short calls store, in which a warp takes one head; some tokens against the oracle's encoder
    page, rng = 64, np.random.default_rng(10)
    n = np.diff(np.sort(np.concatenate([[0, tokens], rng.integers(0, tokens, 4)])))
    n = np.append(n, 0)
    start = rng.integers(0, 100, len(n)).astype(np.int32)
    counts = [(int(s + x) + page - 1) // page for s, x in zip(start, n)]
    cache, signs = new_cache(sum(counts) + 1, heads, page, fill=11)
    same = kv.PagedCache.wrap(cache.pages.clone(), cache.signs)
    before = cache.pages.clone()
    table, _ = table_for(counts, sum(counts) + 1, rng)
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    assert (tokens // 8 + 2 * len(n)) * heads >= 2 * 148 * 28
    g = torch.Generator(device="cuda").manual_seed(12)
    qkv = torch.randn((tokens, q_heads + 2 * heads, 128), generator=g, device="cuda").to(dtype)
    q, k, v = qkv[:, :q_heads], qkv[:, q_heads:q_heads + heads], qkv[:, q_heads + heads:]
    kw, rope_np, pos = {}, None, None
    if rot:
        cs = rope_table(500, rot)
        pos = rng.integers(0, 500, (len(sections), tokens)).astype(np.int32)
        kw = dict(rope=kv.Rope(dev(cs), sections=sections, interleaved=interleaved))
        rope_np = (cs, sections, interleaved)
    tab = dev(table)
    got = cache.append(k, v, tab, dev(start), dev(cu), q=q, positions=dev(pos) if rot else None, **kw)
    part = 8288 // heads * 4      # tokens of a call that gives a warp one head
    want = torch.empty_like(got)
    for b in range(len(n)):
        for t0 in range(cu[b], cu[b + 1], part):
            t1 = min(t0 + part, cu[b + 1])
            assert (-(-(t1 - t0) // 8) + 2) * heads < 2 * 148 * 28
            at = dict(positions=dev(pos[:, t0:t1])) if rot else {}
            want[t0:t1] = same.append(k[t0:t1], v[t0:t1], tab[b:b + 1], dev([start[b] + t0 - cu[b]], torch.int32),
                                      dev([0, t1 - t0], torch.int32), q=q[t0:t1], **at, **kw)
    assert cache.status() == 0 and same.status() == 0
    assert torch.equal(cache.pages, same.pages) and torch.equal(got, want)
    # single tokens: the first and last of a sequence, some between
    after, before = cache.pages.cpu().numpy(), before.cpu().numpy()
    for b in range(len(n)):
        for t in {int(cu[b]), int(cu[b + 1]) - 1, int(cu[b] + n[b] // 2)} if n[b] else ():
            p = int(start[b]) + t - int(cu[b])
            page_no, off = table[b, p // page], p % page
            one = ref.append(before, ref.to_np(k[t:t + 1]), ref.to_np(v[t:t + 1]), table[b:b + 1], [p], [0, 1], signs, rope_np,
                             pos[:, t:t + 1] if rot else None)
            blk, tok = off // 32, off % 32
            for h in {0, heads // 2, heads - 1}:
                a, w = ref.fields(after[page_no, h, blk]), ref.fields(one[page_no, h, blk])
                assert (a[0][ref.bit_row(tok)] == w[0][ref.bit_row(tok)]).all() and a[1][tok] == w[1][tok]
                assert (a[2][:, tok] == w[2][:, tok]).all() and (a[3][:, tok] == w[3][:, tok]).all()
                mask = np.uint32(15) << np.uint32(4 * ref.nibble(tok))
                assert ((a[4][:, tok // 8] & mask) == (w[4][:, tok // 8] & mask)).all()
            for hq in {0, q_heads - 1}:
                row = ref.to_np(q[t, hq])[None]
                row = ref.turn(row, rope_np[0], [pos[a][t] for a in range(len(sections))], sections, interleaved) if rot else row
                assert torch.equal(got[t, hq].cpu(), torch.from_numpy(row[0]).to(dtype))


# ------------------------------------------------------------------------- results beside and over their inputs
def row_elements(offset, T, st, H, sh):
    return (offset + np.arange(T)[:, None, None] * st + np.arange(H)[None, :, None] * sh + np.arange(128)).ravel()


def test_append_refuses_query_rows_that_meet():
    # layouts drawn at random inside one buffer, with what shares an element counted out element by element
    rng = np.random.default_rng(13)
    buf = torch.randn((1 << 16,), device="cuda", dtype=torch.float16)
    cache, _ = new_cache(4, 2, 32)
    seen = {True: 0, False: 0}
    for trial in range(600):
        T, H = int(rng.integers(1, 5)), int(rng.integers(1, 5))
        near = lambda x: int(x + 8 * rng.choice([0, 0, 0, -1, 1, -8, 8]))  # noqa: E731
        if rng.random() < 0.6:
            sh = max(0, near(128 * rng.integers(1, 3)))
            st = max(0, near(sh * int(rng.choice([H, 2 * H, 3 * H]))))
        else:
            st = max(0, near(128 * rng.integers(1, 3)))
            sh = max(0, near(st * int(rng.choice([T, 2 * T]))))
        o0 = 8 * int(rng.integers(0, 1024))
        how = rng.random()
        q0, qst, qsh = o0 + int(rng.choice([0, 128, -128, sh, st, H * sh, 8, 64, 2 * st + sh, 4096])), st, sh
        if how < 0.2:
            qst, qsh = int(rng.choice([0, 128, 256, 512])), int(rng.choice([0, 128, 384]))
        kv0 = o0 + int(rng.choice([8192, 8192, 8192, H * sh, -2 * sh, 64]))
        if min(q0, kv0) < 0:
            continue
        view = lambda at, t, n, h: buf.as_strided((T, n, 128), (t, h, 1), at)  # noqa: E731
        out, q, k = view(o0, st, H, sh), view(q0, qst, H, qsh), view(kv0, st, 2, sh)
        mine = row_elements(o0, T, st, H, sh)
        others = row_elements(kv0, T, st, 2, sh)
        same = q0 == o0 and (T == 1 or qst == st) and (H == 1 or qsh == sh)
        if not same:
            others = np.concatenate([others, row_elements(q0, T, qst, H, qsh)])
        meet = len(np.unique(mine)) < len(mine) or len(np.intersect1d(mine, others)) > 0
        nested = T == 1 or H == 1 or st >= (H - 1) * sh + 128 or sh >= (T - 1) * st + 128
        agree = nested and (same or T == 1 or H == 1 or (qst, qsh) == (st, sh)) and \
            (T == 1 or st >= max((H - 1) * sh, sh) + 128 or H == 2) and how >= 0.2
        call = lambda: cache.append(k, k, dev([[0]], torch.int32), dev([0], torch.int32), dev([0, T], torch.int32), q=q, q_out=out)  # noqa: E731
        expect, before = q.clone(), buf.clone()
        try:
            call()
        except kv.Kv1bError as e:
            assert e.code == -1 and torch.equal(buf, before)
            assert meet or not agree, (T, H, st, sh, o0, q0, qst, qsh, kv0)
            seen[True] += 1
        else:
            assert not meet, (T, H, st, sh, o0, q0, qst, qsh, kv0)
            assert torch.equal(out, expect)
            rest = torch.ones_like(buf, dtype=torch.bool)
            rest[dev(mine)] = False
            assert torch.equal(buf[rest], before[rest])
            seen[False] += 1
    assert min(seen.values()) > 100, seen
    # what serving code does: a slice turned in place, into a neighbouring slice, and transposed
    qkv = torch.randn((6, 12, 128), device="cuda", dtype=torch.float16)
    args = (qkv[:, 8:10], qkv[:, 10:], dev([[0]], torch.int32), dev([0], torch.int32), dev([0, 6], torch.int32))
    rope = dict(rope=kv.Rope(dev(rope_table(64, 128))), positions=torch.arange(6, dtype=torch.int32, device="cuda"))
    want = cache.append(*args, q=qkv[:, :4], **rope)
    cache.append(*args, q=qkv[:, :4], q_out=qkv[:, 4:8], **rope)
    assert torch.equal(qkv[:, 4:8], want)
    turned = torch.empty((4, 6, 128), device="cuda", dtype=torch.float16).transpose(0, 1)
    assert torch.equal(cache.append(*args, q=qkv[:, :4], q_out=turned, **rope), want)
    cache.append(*args, q=qkv[:, :4], q_out=qkv[:, :4], **rope)
    assert torch.equal(qkv[:, :4], want)
    for bad in (qkv[:, 1:5], qkv[:, 5:9], qkv[:, 7:11]):
        with pytest.raises(kv.Kv1bError):
            cache.append(*args, q=qkv[:, :4], q_out=bad, **rope)
    assert cache.status() == 0


def test_one_row_for_all():
    # text through a three-axis model: positions.expand; samples of one sequence: one page list for all
    lengths = [200] * 9
    cache, signs, table, _ = filled([200], 64, 2, 49)
    one = dev(table)
    q = torch.randn((9, 4, 128), device="cuda", dtype=torch.float16)
    n = dev(lengths, torch.int32)
    out = cache.attend(q, SCALE, one.expand(9, -1), n)
    assert torch.equal(out, cache.attend(q, SCALE, one.repeat(9, 1), n))
    check_attend(out, q, cache, signs, SCALE, np.tile(table, (9, 1)), lengths)
    args = (one[0, :1], dev([30], torch.int32))
    shared = cache.attend_shared(q, SCALE, *args, one.expand(9, -1), n)
    assert torch.equal(shared, cache.attend_shared(q, SCALE, *args, one.repeat(9, 1), n))
    rope = kv.Rope(dev(rope_table(300, 96)), sections=[16, 16, 16])
    for tokens in (1, 40):
        k, v, x = torch.randn((3, tokens, 2, 128), device="cuda", dtype=torch.float16)
        pos = torch.randint(0, 300, (tokens,), dtype=torch.int32, device="cuda")
        place = (one, dev([0], torch.int32), dev([0, tokens], torch.int32))
        a = cache.append(k, v, *place, rope=rope, positions=pos.expand(3, tokens), q=x)
        first = cache.pages.clone()
        cache.pages.view(torch.int32).random_()
        cache.pages[table[0]] = 0
        b = cache.append(k, v, *place, rope=rope, positions=pos.repeat(3, 1), q=x)
        assert torch.equal(a, b)
        got, want = ref.fields(cache.pages.cpu().numpy()), ref.fields(first.cpu().numpy())
        rows = [ref.bit_row(t) for t in range(min(tokens, 32))]
        assert (got[0][table[0, 0], :, 0][:, rows] == want[0][table[0, 0], :, 0][:, rows]).all()
    with pytest.raises(kv.Kv1bError):
        cache.append(k[:9], v[:9], one.expand(9, -1), n, dev(range(10), torch.int32))
    assert cache.status() == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("low_halves", [False, True])
def test_results_at_the_end_of_binary16_stay_finite(low_halves, dtype):
    # values at both ends of binary16, and equal weights that are rounded all one way against the sum they are divided by:
    # with low_halves a reference set by 64 lower tokens and 64 higher ones after them in each tile
    n, H, G, B = 9000, 8, 4, 40
    cache, signs, pages, q1 = sized_cache(n, H, 1.0, 0.0)
    share = torch.full((n, 1, 1), 0.2, device="cuda")
    v = torch.full((n, H, 128), 65504.0, device="cuda")
    if low_halves:
        share[torch.arange(n, device="cuda") % 128 < 64] = 0.05
        v[:, :, 32:64] = v[:, :, 96:] = -65504.0
    else:
        share[:64] *= 2
        v[:, :, 1::2] = -65504.0
    cache.append(share * q1, v, dev(pages[None]), dev([0], torch.int32), dev([0, n], torch.int32))
    stored = ref.gather(cache.pages.cpu().numpy(), pages, 0, np.arange(n))[1]
    assert (stored == stored[:1]).all()  # 65504, or 65416 where a group has both ends: min + 15 steps of 8728
    q = (torch.linspace(0.1, 0.75 if low_halves else 2, B, device="cuda")[:, None, None, None] * q1[None, :, None].expand(B, H, G, 128)).reshape(B, H * G, 128)
    wide = np.full((40000 // 64,), -1, np.int32)
    wide[:len(pages)] = pages
    tab, none, full, x = dev(np.tile(pages, (B, 1))), dev([0] * B, torch.int32), dev([n] * B, torch.int32), q.to(dtype)
    for out in (cache.attend_shared(x, SCALE, dev(wide), dev([n], torch.int32), tab, none), cache.attend(x, SCALE, tab, full),
                cache.attend_shared(x, SCALE, dev(wide[:2]), dev([128], torch.int32), tab[:, 2:].contiguous(), full - 128)):
        assert torch.isfinite(out).all()
        # a rounding of the weights against their sum, one of weight scale (a group's values span twice its result at
        # most), fp32 sums, and the result's type
        tol = 2.0 ** -11 + 2 * 2.0 ** -11 + 2.0 ** -18 + torch.finfo(dtype).eps / 2
        assert np.abs(out.double().cpu().numpy() / stored[0] - 1).max() <= tol
    assert cache.status() == 0


# ------------------------------------------------------------------------------------------- wide batches
@pytest.mark.parametrize("tokens", [1000, 3000])
def test_append_to_a_thousand_sequences(tokens):
    # both forms find a token's sequence among 1,000, many of which bring none; query rows turned along
    rng = np.random.default_rng(14)
    n = rng.multinomial(tokens, rng.dirichlet(np.full(1000, 0.3)))
    n[[0, 999]] = 0
    T = int(n.sum())
    start = rng.integers(0, 40, 1000).astype(np.int32)
    counts = [(int(s + x) + 31) // 32 for s, x in zip(start, n)]
    cache, signs = new_cache(sum(counts) + 1, 1, 32, fill=15)
    table, _ = table_for(counts, sum(counts) + 1, rng)
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    k, v, q = torch.randn((3, T, 1, 128), device="cuda", dtype=torch.bfloat16)
    cs, pos = rope_table(200, 128), rng.integers(0, 200, (1, T)).astype(np.int32)
    before = cache.pages.cpu().numpy()
    got = cache.append(k, v, dev(table), dev(start), dev(cu), rope=kv.Rope(dev(cs)), positions=dev(pos), q=q)
    want = ref.append(before, ref.to_np(k), ref.to_np(v), table, start, cu, signs, (cs, [64], False), pos)
    same_bytes(cache.pages.cpu().numpy(), want)
    for t in rng.integers(0, T, 50):
        row = ref.turn(ref.to_np(q[t]), cs, [pos[0, t]], [64], False)
        assert torch.equal(got[t].cpu(), torch.from_numpy(row).to(q.dtype))
    assert cache.status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens", [2, 61])
def test_append_sections_of_any_size(tokens, interleaved, dtype):
    # axes that change inside four pairs, an axis without pairs, keys and values spread over heads or tokens by strides
    rng = np.random.default_rng(16)
    for sections in ([11, 27, 26], [1, 0, 63], [0, 63, 1], [5, 8, 7], [0, 0, 4]):
        rot = 2 * sum(sections)
        cache, signs = new_cache(4, 3, 64, fill=17)
        cs, pos = rope_table(90, rot), rng.integers(0, 90, (3, tokens)).astype(np.int32)
        k = torch.randn((3, tokens, 128), device="cuda").to(dtype).transpose(0, 1)
        v = torch.randn((tokens, 1, 128), device="cuda").to(dtype).expand(tokens, 3, 128)
        q = torch.randn((5, tokens, 132), device="cuda").to(dtype)[:, :, :128].transpose(0, 1)
        table = np.array([[2, 1]], np.int32)
        before = cache.pages.cpu().numpy()
        rope = kv.Rope(dev(cs), sections=sections, interleaved=interleaved)
        got = cache.append(k, v, dev(table), dev([50], torch.int32), dev([0, tokens], torch.int32), rope=rope, positions=dev(pos), q=q)
        want = ref.append(before, ref.to_np(k), ref.to_np(v), table, [50], [0, tokens], signs, (cs, sections, interleaved), pos)
        same_bytes(cache.pages.cpu().numpy(), want, f"sections {sections}")
        for t in range(tokens):
            row = ref.turn(ref.to_np(q[t]), cs, pos[:, t], sections, interleaved)
            assert torch.equal(got[t].cpu(), torch.from_numpy(row).to(dtype)), (sections, t)


def test_attend_shared_a_thousand_sequences():
    # 2,048 rows of a kv-head: eight row tiles, each over the whole prefix
    rng = np.random.default_rng(18)
    lengths, prefix = [int(x) for x in rng.integers(0, 33, 1024)], 333
    cache, signs, table, pre = filled(lengths, 32, 2, 50, prefix=prefix, width=1)
    q = (2 * torch.randn((1024, 4, 128), device="cuda")).to(torch.bfloat16)
    args = (q, SCALE, dev(pre), dev([prefix], torch.int32), dev(table), dev(lengths, torch.int32))
    out = cache.attend_shared(*args)
    assert cache.status() == 0 and torch.equal(out, cache.attend_shared(*args))
    check_rows(out, q, cache, signs, SCALE, table, lambda b: np.arange(lengths[b]), some_rows(rng, 1024, 4, 200),
               prefix=(pre, np.arange(prefix)))


@pytest.mark.parametrize("cu", [[0, 100, 3, 8], [0, 9, 9, 200], [-1, 3, 5, 9], [0, 60, 59, 120]])
@pytest.mark.parametrize("copies", [1, 20])
def test_append_reports_rows_that_do_not_ascend(cu, copies):
    # wherever the fault is, also at a sequence that no row leads to; both forms, few and many sequences; nothing is
    # written outside the sequences' places
    cu = np.concatenate([np.array(cu)] + [np.array(cu[-1:] * 3)] * (copies - 1))
    B, T = len(cu) - 1, 120
    for tokens in (T, B + 1):
        cache, _ = new_cache(5 * B + 2, 1, 32, fill=19)
        table, spare = table_for([5] * B, 5 * B + 2, np.random.default_rng(20))
        k = torch.randn((tokens, 1, 128), device="cuda", dtype=torch.float16)
        before = cache.pages.cpu().numpy()
        cache.append(k, k, dev(table), dev([0] * B, torch.int32), dev(cu, torch.int32))
        assert cache.status() == kv.STATUS_BAD_INDEX
        after = cache.pages.cpu().numpy()
        same_bytes(after[spare], before[spare])
        same_bytes(after[table[:, 4]], before[table[:, 4]])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rounds", [1, 2, 3])
@pytest.mark.parametrize("group, page", [(3, 32), (7, 256), (8, 4096)])
def test_attend_after_several_rotation_rounds(rounds, group, page, dtype):
    # the queries' side of every kernel with 1 to 3 rounds, odd groups, the smallest and the largest page
    n, H, B = 700, 2, 50
    num = (n + page - 1) // page
    cache, signs = new_cache(num + 1, H, page, rounds=rounds, seed=21)
    k, v = torch.randn((2, n, H, 128), device="cuda")
    pages = np.random.default_rng(21).permutation(num).astype(np.int32)
    cache.append(k, v, dev(pages[None]), dev([0], torch.int32), dev([0, n], torch.int32))
    q = (2 * torch.randn((B, H * group, 128), device="cuda")).to(dtype)
    table, lengths = np.tile(pages, (B, 1)), [int(x) for x in np.linspace(0, n, B)]
    rows = some_rows(np.random.default_rng(22), B, H * group, 20)
    tab, count = dev(table), dev(lengths, torch.int32)
    out = cache.attend(q, SCALE, tab, count)
    check_rows(out, q, cache, signs, SCALE, table, lambda b: np.arange(lengths[b]), rows)
    # 4 rows a kv-head and fewer in the attend's kernel, 150 and more in the matrix kernel
    for some in (slice(0, 1), slice(0, B)):
        out = cache.attend_shared(q[some], SCALE, dev(pages), dev([n], torch.int32), tab[some], count[some])
        check_rows(out, q[some], cache, signs, SCALE, table, lambda b: np.arange(lengths[b]),
                   [r for r in rows if r[0] < len(out)] + [(0, 1)], prefix=(pages, np.arange(n)))
    assert cache.status() == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_fp16_rows_that_are_not_finite_stay_so(bad):
    # the limit of fp16 results hides no NaN: spoilt queries' rows, all of them and no others, in the three kernels
    lengths, prefix, page = [90, 5, 33, 700] * 12, 300, 64
    cache, signs, table, pre = filled(lengths, page, 2, 51, prefix=prefix)
    q = torch.randn((48, 8, 128), device="cuda", dtype=torch.float16)
    q[1, 2, 77] = bad
    q[3, 5] = bad
    q[13, 0, :] = bad
    spoilt = torch.zeros((48, 8), dtype=torch.bool, device="cuda")
    spoilt[1, 2] = spoilt[3, 5] = spoilt[13, 0] = True
    tab, n, plen = dev(table), dev(lengths, torch.int32), dev([prefix], torch.int32)
    for out in (cache.attend(q, SCALE, tab, n), cache.attend_shared(q, SCALE, dev(pre), plen, tab, n),
                cache.attend_shared(q[:4], SCALE, dev(pre), plen, tab[:4], n[:4])):
        assert torch.equal(torch.isfinite(out).all(-1), ~spoilt[:len(out)])
        assert torch.equal(torch.isfinite(out).any(-1), ~spoilt[:len(out)])
