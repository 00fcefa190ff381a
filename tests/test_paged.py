"""The paged cache on the GPU: the append against the oracle's encoder byte for byte (untouched bytes
included), attention against 64 bits, and the calls together as a serving loop makes them."""
import concurrent.futures

import numpy as np
import pytest
import torch

import oracle
import long_context_decode_kv1b_b200 as kv
import paged_reference as ref

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(20)


def table_for(counts, num_pages, rng, width=None):
    """Shuffled pages: int32 [seqs, width], -1 behind a sequence's pages."""
    order = rng.permutation(num_pages)
    width = width or max(max(counts), 1)
    out, at = -np.ones((len(counts), width), np.int32), 0
    for b, c in enumerate(counts):
        out[b, :c] = order[at:at + c]
        at += c
    assert at <= num_pages
    return out, order[at:].astype(np.int32)


def dev(a, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=dtype, device="cuda")


def rope_table(n, rot):
    half = rot // 2
    ang = np.arange(n)[:, None] * 1e4 ** (-np.arange(half) / half)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def new_cache(num_pages, heads, page_tokens, rounds=1, seed=3, fill=None):
    c = kv.PagedCache(num_pages, heads, page_tokens, seed=seed, rounds=rounds)
    if fill is not None:
        g = torch.Generator(device="cuda").manual_seed(fill)
        c.pages.view(torch.int32).random_(-2 ** 31, 2 ** 31 - 1, generator=g)
    return c, oracle.signs(seed, rounds=rounds)


def same_bytes(got, want, what=""):
    bad = np.argwhere(got != want)
    assert len(bad) == 0, f"{what}: {len(bad)} bytes differ, first {bad[:4].tolist()}"


# ------------------------------------------------------------------------------------------ append
# (new tokens per sequence, tokens held, page, heads, group, rot, sections, interleaved, rounds)
APPENDS = [
    ([1], [0], 32, 1, 1, 128, [64], False, 1),
    ([1, 1, 1], [5, 31, 32], 64, 3, 2, 128, [64], False, 1),
    ([1] * 40, list(range(40)), 32, 2, 1, 64, [32], True, 1),
    ([0, 2, 1, 0, 4], [7, 63, 64, 0, 30], 64, 2, 4, 96, [16, 16, 16], False, 3),
    ([75], [13], 128, 2, 3, 128, [64], False, 2),
    ([40, 0, 1, 66, 9], [0, 3, 31, 250, 8], 64, 2, 1, 128, [16, 24, 24], False, 1),
    ([33, 64], [1, 96], 32, 5, 1, 32, [16], True, 1),
    ([50], [6], 256, 1, 8, 8, [4], False, 1),
    ([37, 20], [64, 2], 64, 2, 2, 0, [], False, 1),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("case", range(len(APPENDS)))
def test_append_bytes(case, dtype):
    n, start, page, H, G, rot, sections, inter, rounds = APPENDS[case]
    rng = np.random.default_rng(100 + case)
    counts = [(s + x + page - 1) // page for s, x in zip(start, n)]
    num_pages = sum(counts) + 2
    cache, signs = new_cache(num_pages, H, page, rounds, fill=case + 1)
    table, _ = table_for(counts, num_pages, rng)
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    pad = 3                                       # rows behind the last sequence
    T = int(cu[-1]) + pad
    g = torch.Generator(device="cuda").manual_seed(case)
    qkv = torch.randn((T, H * G + 2 * H, 128), generator=g, device="cuda").to(dtype)
    q, k, v = qkv[:, :H * G], qkv[:, H * G:H * G + H], qkv[:, H * G + H:]
    v[0, 0, :32] = 0.25
    k[T - pad - 1, 0] = 0
    rope = pos = rope_np = pos_np = None
    if rot:
        cs = rope_table(400, rot)
        pos_np = rng.integers(0, 400, (len(sections), T)).astype(np.int32)
        rope, pos = kv.Rope(dev(cs), sections=sections, interleaved=inter), dev(pos_np)
        rope_np = (cs, sections, inter)
    before = cache.pages.cpu().numpy()
    q_out = torch.full_like(q, 7.0)
    got = cache.append(k, v, dev(table), dev(start, torch.int32), dev(cu), rope=rope, positions=pos, q=q, q_out=q_out)
    assert got is q_out
    want = ref.append(before, ref.to_np(k), ref.to_np(v), table, start, cu, signs, rope_np, pos_np)
    same_bytes(cache.pages.cpu().numpy(), want, f"pages of case {case}")
    qn = ref.to_np(q)
    for t in range(T):
        if t >= cu[-1]:
            assert (q_out[t] == 7.0).all()
            continue
        row = ref.turn(qn[t], rope_np[0], [pos_np[a][t] for a in range(len(sections))], sections, inter) if rot else qn[t]
        assert torch.equal(q_out[t].cpu(), torch.from_numpy(row).to(dtype)), f"q row {t}"
    assert cache.status() == 0


def test_append_in_place_query_and_one_dimensional_positions():
    cache, _ = new_cache(2, 1, 64, fill=2)
    cs = rope_table(64, 128)
    rope = kv.Rope(dev(cs))
    q = torch.randn((5, 2, 128), device="cuda", dtype=torch.float16)
    k = torch.randn((5, 1, 128), device="cuda", dtype=torch.float16)
    args = (k, k, dev([[0]], torch.int32), dev([0], torch.int32), dev([0, 5], torch.int32))
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    a = cache.append(*args, rope=rope, positions=pos, q=q)
    b = cache.append(*args, rope=rope, positions=pos[None], q=q, q_out=q)
    assert b is q and torch.equal(a, b)


@pytest.mark.parametrize("tokens", [3, 90])
def test_append_extreme_values(tokens):
    # fp32 values past the binary16 range are limited, the top code stays inside it, NaN counts as 0
    cache, signs = new_cache(3, 2, 64, fill=9)
    k = torch.randn((tokens, 2, 128), device="cuda")
    v = torch.randn((tokens, 2, 128), device="cuda")
    v[0, 0, :64] *= 1e6
    v[1, 1, 5] = -65504.0
    v[1, 1, 6] = 65504.0
    v[2, 0] = 3.4e38
    table = np.array([[2, 0]], np.int32)
    before = cache.pages.cpu().numpy()
    call = lambda: cache.append(k, v, dev(table), dev([0], torch.int32), dev([0, tokens], torch.int32))  # noqa: E731
    call()
    assert cache.status() == kv.STATUS_FP16_SATURATED
    want = ref.append(before, ref.to_np(k), ref.to_np(v), table, [0], [0, tokens], signs)
    same_bytes(cache.pages.cpu().numpy(), want)
    _, nc, scale, least, _ = ref.fields(cache.pages.cpu().numpy())
    used = np.isin(np.arange(3), table[0, :(tokens + 63) // 64])
    halves = [x[used][:, :, 0, :, :3].view(np.float16).astype(float) for x in (least, scale)]
    top = halves[0] + 15.0 * halves[1]
    assert (np.abs(top) <= 65504).all()
    v[1, 0, 3] = float("nan")
    before = cache.pages.cpu().numpy()
    call()
    assert cache.status() & kv.STATUS_NONFINITE
    same_bytes(cache.pages.cpu().numpy(), ref.append(before, ref.to_np(k), ref.to_np(v), table, [0], [0, tokens], signs))


@pytest.mark.parametrize("per_seq", [1, 40])
def test_append_skips_what_has_no_place(per_seq):
    # a page past the cache, a negative one, a position outside the rotary table, a table too short
    n = [per_seq] * 5
    cache, signs = new_cache(8, 2, 32, fill=4)
    table = np.array([[0, 1], [99, 2], [-1, 3], [4, 5], [6, 7]], np.int32)
    start = [0, 0, 3, 0, 60]
    cu = np.arange(6, dtype=np.int32) * per_seq
    T = 5 * per_seq
    k, v = torch.randn((2, T, 2, 128), device="cuda", dtype=torch.bfloat16)
    cs = rope_table(50, 64)
    pos = np.tile(np.arange(T, dtype=np.int32) % 50, (1, 1))
    pos[0, 3 * per_seq] = 50
    before = cache.pages.cpu().numpy()
    cache.append(k, v, dev(table), dev(start, torch.int32), dev(cu), rope=kv.Rope(dev(cs)), positions=dev(pos))
    assert cache.status() == kv.STATUS_BAD_INDEX
    same_bytes(cache.pages.cpu().numpy(),
               ref.append(before, ref.to_np(k), ref.to_np(v), table, start, cu, signs, (cs, [32], False), pos))
    # a sequence whose start is negative, or whose rows are out of order, is left out whole
    cache.status_word.zero_()
    before = cache.pages.cpu().numpy()
    cache.append(k, v, dev(table), dev([-1, 0, 0, 0, 0], torch.int32), dev([0] + [per_seq] * 5, torch.int32))
    assert cache.status() == kv.STATUS_BAD_INDEX
    same_bytes(cache.pages.cpu().numpy(), before)


# ------------------------------------------------------------------------------------------ attend
def filled(lengths, page, H, seed, prefix=None, spare=2, width=None):
    """A cache whose sequences hold `lengths` tokens; every other byte is random, the other tokens'
    scalars NaN and infinities among them."""
    rng = np.random.default_rng(seed)
    counts = [(n + page - 1) // page for n in lengths]
    npre = 0 if prefix is None else (prefix + page - 1) // page
    num = sum(counts) + npre + spare
    cache, signs = new_cache(num, H, page, fill=seed)
    table, rest = table_for(counts, num, rng, width)
    g = torch.Generator(device="cuda").manual_seed(seed)
    runs = [(table[b], n) for b, n in enumerate(lengths)] + ([(rest[:npre], prefix)] if npre else [])
    for row, n in runs:
        if n:
            k, v = torch.randn((2, n, H, 128), generator=g, device="cuda", dtype=torch.bfloat16)
            cache.append(k, v, dev(row[None]), dev([0], torch.int32), dev([0, n], torch.int32))
            last = row[(n - 1) // page]          # poison behind the last token
            off = (n - 1) % page
            blk, tok = off // 32, off % 32
            raw = cache.pages[int(last)]
            for b in range(blk, page // 32):
                lo = tok + 1 if b == blk else 0
                raw[:, b, 512:640].view(torch.float32)[:, lo:] = float("nan")
                for at in (640, 896):
                    f = raw[:, b, at:at + 256].view(torch.float16).view(H, 4, 32)
                    f[:, :, lo::2], f[:, :, lo + 1::2] = float("inf"), float("nan")
    assert cache.status() == 0
    return cache, signs, table, rest[:npre].astype(np.int32)


def check_attend(out, q, cache, signs, scale, table, lengths, window=0, sinks=0, prefix=None, rows=None):
    pages, qn, got = cache.pages.cpu().numpy(), ref.to_np(q), ref.to_np(out).astype(np.float64)
    G = q.shape[1] // cache.num_kv_heads
    eps = torch.finfo(q.dtype).eps
    for b in range(len(lengths)):
        n = lengths[b]
        t = np.arange(n)
        if window:
            t = t[(t >= n - window) | (t < sinks)]
        for h in range(cache.num_kv_heads):
            parts = [ref.gather(pages, table[b], h, t)]
            if prefix is not None:
                parts.insert(0, ref.gather(pages, prefix[0], h, np.arange(prefix[1])))
            for r in range(G):
                row = ref.Row(qn[b, h * G + r], signs, scale, parts)
                tol = row.tolerance(eps)
                err = np.abs(got[b, h * G + r] - row.out)
                assert (err <= tol).all(), f"seq {b} (length {n}) head {h}.{r}: error {err.max():.3e}, " \
                                           f"{(err / tol).max():.2f} of the tolerance"


ATTENDS = [
    # lengths, page, kv heads, group, window, sinks
    ([1], 32, 1, 1, 0, 0),
    ([0, 1, 31, 32, 33, 0], 32, 2, 3, 0, 0),
    ([397], 128, 8, 4, 0, 0),
    ([700, 1, 0, 129, 64, 1000], 64, 2, 5, 0, 0),
    ([2000, 313], 256, 1, 8, 0, 0),
    ([1500], 128, 3, 7, 0, 0),
    ([5, 200, 1, 0, 333], 32, 2, 2, 1, 0),
    ([100, 31, 32, 33, 700], 64, 2, 4, 33, 5),
    ([640, 65, 66], 64, 1, 8, 64, 64),
    ([900, 64], 128, 2, 6, 500, 33),
    ([300, 299], 64, 2, 4, 200, 250),      # sinks reach into the window
    ([90, 3], 32, 2, 1, 1000, 7),           # windows longer than the sequence
    ([97] * 130, 32, 1, 2, 0, 0),           # more sequences than a small plan has CTAs for
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", range(len(ATTENDS)))
def test_attend(case, dtype):
    lengths, page, H, G, window, sinks = ATTENDS[case]
    cache, signs, table, _ = filled(lengths, page, H, 50 + case)
    q = (2 * torch.randn((len(lengths), H * G, 128), device="cuda")).to(dtype)
    out = cache.attend(q, SCALE, dev(table), dev(lengths, torch.int32), window=window, sinks=sinks)
    assert out.dtype == dtype and cache.status() == 0
    check_attend(out, q, cache, signs, SCALE, table, lengths, window, sinks)
    for b, n in enumerate(lengths):
        if n == 0:
            assert (out[b] == 0).all()


@pytest.mark.parametrize("scale", [0.0, 3.0, -1.0])
def test_attend_flat_and_peaked(scale):
    # every token alike, one token alone, and the order turned round
    lengths = [260, 513]
    cache, signs, table, _ = filled(lengths, 128, 2, 8)
    q = torch.randn((2, 4, 128), device="cuda", dtype=torch.float16)
    out = cache.attend(q, scale, dev(table), dev(lengths, torch.int32))
    check_attend(out, q, cache, signs, scale, table, lengths)


def test_attend_rising_logits():
    # keys that point ever more at the query: the running reference is raised again and again
    n, page = 640, 64
    cache, signs = new_cache(10, 1, page)
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn((1, 1, 128), generator=g, device="cuda", dtype=torch.bfloat16)
    k = (torch.linspace(0, 8, n, device="cuda")[:, None, None] * q.float() + 0.3 * torch.randn((n, 1, 128), generator=g, device="cuda"))
    v = torch.randn((n, 1, 128), generator=g, device="cuda")
    table = np.arange(10, dtype=np.int32)[None]
    cache.append(k, v, dev(table), dev([0], torch.int32), dev([0, n], torch.int32))
    for scale in (SCALE, 4 * SCALE):
        out = cache.attend(q, scale, dev(table), dev([n], torch.int32))
        check_attend(out, q, cache, signs, scale, table, [n])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("size", [1e-4, 30.0, 2000.0, 65504.0])
def test_attend_small_and_large_values(size, dtype):
    # value scales from subnormal to the largest, growing along the sequence and within one block
    n, page = 400, 64
    cache, signs = new_cache(7, 2, page)
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = torch.randn((2, n, 2, 128), generator=g, device="cuda")
    v *= size * torch.linspace(1e-3, 1, n, device="cuda")[:, None, None]
    v[37, 0, :32] = size * torch.linspace(-1, 1, 32, device="cuda")
    v.clamp_(-65504, 65504)
    table = np.arange(7, dtype=np.int32)[None]
    cache.append(k, v, dev(table), dev([0], torch.int32), dev([0, n], torch.int32))
    q = torch.randn((1, 8, 128), generator=g, device="cuda").to(dtype)
    out = cache.attend(q, SCALE, dev(table), dev([n], torch.int32))
    check_attend(out, q, cache, signs, SCALE, table, [n])
    out = cache.attend_shared(q, SCALE, dev(table[0, :3]), dev([192], torch.int32), dev(table[:, 3:]), dev([n - 192], torch.int32))
    check_attend(out, q, cache, signs, SCALE, table, [n])


def test_attend_bad_pages_and_lengths():
    # entries outside the cache count as unseen, lengths are limited to the table, both are reported
    lengths = [200, 150]
    cache, signs, table, _ = filled(lengths, 32, 2, 21)
    q = torch.randn((2, 4, 128), device="cuda", dtype=torch.float16)
    bad = table.copy()
    bad[0, 2], bad[1, 0] = cache.num_pages, -5
    out = cache.attend(q, SCALE, dev(bad), dev(lengths, torch.int32))
    assert cache.status() == kv.STATUS_BAD_INDEX
    pages, qn = cache.pages.cpu().numpy(), ref.to_np(q)
    for b, gone in ((0, 2), (1, 0)):
        t = np.arange(lengths[b])
        t = t[t // 32 != gone]
        row = ref.Row(qn[b, 3], signs, SCALE, [ref.gather(pages, table[b], 1, t)])
        assert (np.abs(ref.to_np(out)[b, 3] - row.out) <= row.tolerance(torch.finfo(q.dtype).eps)).all()
    cache.status_word.zero_()
    out = cache.attend(q, SCALE, dev(np.full_like(table, -1)), dev(lengths, torch.int32))
    assert (out == 0).all() and cache.status() == kv.STATUS_BAD_INDEX
    cache.status_word.zero_()
    out = cache.attend(q, SCALE, dev(table), dev([-3, 150], torch.int32))
    assert cache.status() == kv.STATUS_BAD_INDEX and (out[0] == 0).all()
    check_attend(out[1:], q[1:], cache, signs, SCALE, table[1:], lengths[1:])
    cache.status_word.zero_()
    full = cache.attend(q[:1], SCALE, dev(table[:1, :4]), dev([128], torch.int32))
    more = cache.attend(q[:1], SCALE, dev(table[:1, :4]), dev([2 ** 31 - 1], torch.int32))
    assert cache.status() == kv.STATUS_BAD_INDEX and torch.equal(full, more)


# ------------------------------------------------------------------------------------------ shared
SHARED = [
    # prefix, lengths, page, kv heads, group
    (1, [1, 0], 32, 1, 1),
    (100, [61, 1, 0, 33], 64, 2, 4),
    (1000, [5, 300], 128, 2, 8),
    (0, [40, 7], 32, 2, 3),
    (777, [0, 0, 0], 64, 1, 5),
    (500, [31] * 40, 128, 1, 4),       # more rows than one 128-row tile
    (257, [9] * 33, 256, 2, 8),
    (130, [17] * 300, 32, 1, 1),
    (2100, [70, 0, 5, 33], 64, 3, 8),  # as many rows as the plain kernel packs
    (900, [20] * 11, 64, 2, 3),         # one more than that
    (1500, [3] * 16, 128, 1, 8),        # a full 128-row tile
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", range(len(SHARED)))
def test_attend_shared(case, dtype):
    prefix, lengths, page, H, G = SHARED[case]
    cache, signs, table, pre = filled(lengths, page, H, 80 + case, prefix=prefix)
    if len(pre) == 0:
        pre = np.array([-1], np.int32)
    q = (2 * torch.randn((len(lengths), H * G, 128), device="cuda")).to(dtype)
    out = cache.attend_shared(q, SCALE, dev(pre), dev([prefix], torch.int32), dev(table), dev(lengths, torch.int32))
    assert cache.status() == 0
    check_attend(out, q, cache, signs, SCALE, table, lengths, prefix=(pre, prefix))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows", [17, 32, 33, 64, 128])
@pytest.mark.parametrize("prefix", [0, 1, 100, 900])
def test_attend_shared_wide_prefix_table(prefix, rows, dtype):
    # the same prefix through a table of its own and through one that could hold a long prefix: which kernel
    # takes it follows from the table's width
    lengths, page, H = [29] * rows, 64, 2
    lengths[3:5] = [0, 70]
    cache, signs, table, pre = filled(lengths, page, H, 140 + rows, prefix=prefix)
    if len(pre) == 0:
        pre = np.array([-1], np.int32)
    q = (2 * torch.randn((rows, H, 128), device="cuda")).to(dtype)
    tab, n, plen = dev(table), dev(lengths, torch.int32), dev([prefix], torch.int32)
    near = cache.attend_shared(q, SCALE, dev(pre), plen, tab, n)
    wide = torch.full((70000 * 128 // (page * rows * H),), -1, dtype=torch.int32, device="cuda")
    wide[:len(pre)] = dev(pre)
    far = cache.attend_shared(q, SCALE, wide, plen, tab, n)
    assert cache.status() == 0
    check_attend(near, q, cache, signs, SCALE, table, lengths, prefix=(pre, prefix))
    check_attend(far, q, cache, signs, SCALE, table, lengths, prefix=(pre, prefix))


@pytest.mark.parametrize("prefix, own", [(20000, 200), (20000, 0), (20000, 3), (700, 200)])
def test_attend_shared_own_tokens_beside_the_prefix(prefix, own):
    # few CTAs for the sequences' own tokens while the prefix is worked on; with a short prefix in the same
    # table, many behind it
    lengths, page, H, G = [own - own * (b % 5) // 7 for b in range(40)], 64, 2, 4
    cache, signs, table, pre = filled(lengths, page, H, 150, prefix=20000)
    q = (2 * torch.randn((40, H * G, 128), device="cuda")).to(torch.bfloat16)
    out = cache.attend_shared(q, SCALE, dev(pre), dev([prefix], torch.int32), dev(table), dev(lengths, torch.int32))
    assert cache.status() == 0
    some = [0, 1, 17, 39]
    check_attend(out[some], q[some], cache, signs, SCALE, table[some], [lengths[b] for b in some], prefix=(pre, prefix))


def test_attend_shared_bad_prefix():
    lengths, prefix = [40, 70, 1], 150
    cache, signs, table, pre = filled(lengths, 32, 2, 31, prefix=prefix)
    q = torch.randn((3, 8, 128), device="cuda", dtype=torch.bfloat16)
    args = (dev(table), dev(lengths, torch.int32))
    bad = pre.copy()
    bad[1] = -1
    out = cache.attend_shared(q, SCALE, dev(bad), dev([prefix], torch.int32), *args)
    assert cache.status() == kv.STATUS_BAD_INDEX
    pages, qn = cache.pages.cpu().numpy(), ref.to_np(q)
    t = np.arange(prefix)
    t = t[t // 32 != 1]
    for b in range(3):
        parts = [ref.gather(pages, pre, 1, t), ref.gather(pages, table[b], 1, np.arange(lengths[b]))]
        row = ref.Row(qn[b, 5], signs, SCALE, parts)
        assert (np.abs(ref.to_np(out)[b, 5] - row.out) <= row.tolerance(torch.finfo(q.dtype).eps)).all()
    cache.status_word.zero_()
    out = cache.attend_shared(q, SCALE, dev(pre), dev([-4], torch.int32), *args)
    assert cache.status() == kv.STATUS_BAD_INDEX
    check_attend(out, q, cache, signs, SCALE, table, lengths)


# -------------------------------------------------------------------------------------- together
def test_attend_shared_bad_prefix_in_a_wide_table():
    # the same refusals where the matrix kernel takes the prefix
    lengths, prefix, page = [40, 0] * 20, 700, 32
    cache, signs, table, pre = filled(lengths, page, 2, 33, prefix=prefix)
    q = torch.randn((40, 4, 128), device="cuda", dtype=torch.float16)
    args = (dev(table), dev(lengths, torch.int32))
    wide = np.full((70000 * 128 // (page * 80 * 2),), -1, np.int32)
    wide[:len(pre)] = pre
    wide[[0, 3, 20]] = [cache.num_pages, -9, 2 ** 31 - 1]
    out = cache.attend_shared(q, SCALE, dev(wide), dev([prefix], torch.int32), *args)
    assert cache.status() == kv.STATUS_BAD_INDEX
    pages, qn = cache.pages.cpu().numpy(), ref.to_np(q)
    t = np.arange(prefix)
    t = t[~np.isin(t // page, [0, 3, 20])]
    for b in (0, 1, 39):
        parts = [ref.gather(pages, wide, 1, t), ref.gather(pages, table[b], 1, np.arange(lengths[b]))]
        row = ref.Row(qn[b, 3], signs, SCALE, parts)
        assert (np.abs(ref.to_np(out)[b, 3] - row.out) <= row.tolerance(torch.finfo(q.dtype).eps)).all()
    cache.status_word.zero_()
    out = cache.attend_shared(q, SCALE, dev(wide), dev([-1], torch.int32), *args)
    assert cache.status() == kv.STATUS_BAD_INDEX
    check_attend(out, q, cache, signs, SCALE, table, lengths)
    cache.status_word.zero_()
    out = cache.attend_shared(q, SCALE, dev(np.full_like(wide, -1)), dev([2 ** 31 - 1], torch.int32), *args)
    assert cache.status() == kv.STATUS_BAD_INDEX
    check_attend(out, q, cache, signs, SCALE, table, lengths)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_query_that_is_not_finite_spoils_its_own_row_only(bad):
    lengths, prefix, page = [90, 5, 33, 64] * 6, 300, 64
    cache, signs, table, pre = filled(lengths, page, 2, 34, prefix=prefix)
    q = torch.randn((24, 4, 128), device="cuda", dtype=torch.bfloat16)
    spoilt = q.clone()
    spoilt[1, 2, 77] = bad
    spoilt[13, 0, :] = bad
    ok = torch.ones((24, 4, 1), dtype=torch.bool, device="cuda")
    ok[1, 2] = ok[13, 0] = False
    tab, n, plen = dev(table), dev(lengths, torch.int32), dev([prefix], torch.int32)
    wide = torch.full((70000 * 128 // (page * 48 * 2),), -1, dtype=torch.int32, device="cuda")
    wide[:len(pre)] = dev(pre)

    def patched(out, clean):  # rows of the spoilt queries as those of the clean ones
        assert torch.isfinite(out[ok.expand_as(out)]).all() and not torch.isfinite(out[~ok.expand_as(out)]).any()
        return torch.where(ok, out, clean)

    check_attend(patched(cache.attend(spoilt, SCALE, tab, n), cache.attend(q, SCALE, tab, n)), q, cache, signs, SCALE, table, lengths)
    for pages in (dev(pre), wide):
        out = patched(cache.attend_shared(spoilt, SCALE, pages, plen, tab, n), cache.attend_shared(q, SCALE, pages, plen, tab, n))
        check_attend(out, q, cache, signs, SCALE, table, lengths, prefix=(pre, prefix))


def test_results_over_the_queries():
    # out may be q: one long sequence that every CTA reads, short ones, an empty one, both shared forms
    lengths, prefix, page = [20000, 0, 70, 1] + [33] * 20, 500, 64
    cache, signs, table, pre = filled(lengths, page, 2, 35, prefix=prefix)
    q = torch.randn((24, 4, 128), device="cuda", dtype=torch.float16)
    tab, n, plen = dev(table), dev(lengths, torch.int32), dev([prefix], torch.int32)
    wide = torch.full((70000 * 128 // (page * 48 * 2),), -1, dtype=torch.int32, device="cuda")
    wide[:len(pre)] = dev(pre)
    for call in (lambda x, **kw: cache.attend(x, SCALE, tab, n, **kw),
                 lambda x, **kw: cache.attend_shared(x, SCALE, dev(pre), plen, tab, n, **kw),
                 lambda x, **kw: cache.attend_shared(x, SCALE, wide, plen, tab, n, **kw)):
        apart, same = call(q), q.clone()
        assert call(same, out=same) is same and torch.equal(apart, same)
    k = torch.randn((24, 2, 128), device="cuda", dtype=torch.float16)
    rope = kv.Rope(torch.randn((64, 128), device="cuda"))
    at = torch.arange(24, dtype=torch.int32, device="cuda")
    for _ in range(20):  # a step's append in place, and the attend behind it at once
        same = q.clone()
        turned = cache.append(k, k, tab, n - 1, torch.arange(25, dtype=torch.int32, device="cuda"), rope, at, q=q)
        expect = cache.attend(turned, SCALE, tab, n)
        torch.cuda.synchronize()
        cache.append(k, k, tab, n - 1, torch.arange(25, dtype=torch.int32, device="cuda"), rope, at, q=same, q_out=same)
        assert torch.equal(cache.attend(same, SCALE, tab, n, out=same), expect)


def test_serving_loop_in_graphs():
    # a shared instruction, ragged prompts in chunks, then decode steps replayed from one captured
    # graph while lengths, positions and inputs change in place; a second graph of the same calls is
    # alive meanwhile.  Checked at every step against the oracle's encoder and 64-bit attention.
    H, G, page, B = 2, 4, 32, 3
    cache, signs = new_cache(24, H, page, fill=6)
    rng = np.random.default_rng(6)
    pre = np.array([20, 23], np.int32)
    table, _ = table_for([6, 6, 6], 20, rng, width=6)
    cs = rope_table(512, 128)
    rope = kv.Rope(dev(cs))
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda n, h: torch.randn((n, h, 128), generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    shadow = cache.pages.cpu().numpy()

    def add(k, v, tab, start, cu, pos, q=None):
        nonlocal shadow
        shadow = ref.append(shadow, ref.to_np(k), ref.to_np(v), tab, start, cu, signs, (cs, [64], False), pos)

    k, v = rnd(45, H), rnd(45, H)
    pos = np.arange(45, dtype=np.int32)[None]
    cache.append(k, v, dev(pre[None]), dev([0], torch.int32), dev([0, 45], torch.int32), rope=rope, positions=dev(pos))
    add(k, v, pre[None], [0], [0, 45], pos)
    lengths = [0, 0, 0]
    for chunk in ([20, 1, 33], [9, 0, 12]):
        cu = np.concatenate([[0], np.cumsum(chunk)]).astype(np.int32)
        k, v = rnd(int(cu[-1]), H), rnd(int(cu[-1]), H)
        pos = np.concatenate([45 + s + np.arange(c) for s, c in zip(lengths, chunk)]).astype(np.int32)[None]
        cache.append(k, v, dev(table), dev(lengths, torch.int32), dev(cu), rope=rope, positions=dev(pos))
        add(k, v, table, lengths, cu, pos)
        lengths = [a + b for a, b in zip(lengths, chunk)]
    same_bytes(cache.pages.cpu().numpy(), shadow, "after the prompts")

    k, v, q = rnd(B, H), rnd(B, H), rnd(B, H * G)
    start, cu, pos = dev(lengths, torch.int32), dev(np.arange(B + 1), torch.int32), dev([45 + x for x in lengths], torch.int32)
    after = start + 1
    tab, prefix, plen = dev(table), dev(pre), dev([45], torch.int32)

    def step():
        qr = cache.append(k, v, tab, start, cu, rope=rope, positions=pos, q=q)
        return qr, cache.attend_shared(qr, SCALE, prefix, plen, tab, after), cache.attend(qr, SCALE, tab, after, window=16, sinks=2)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            res = step()
        graphs.append((gr, res))
    for i in range(5):
        k.copy_(rnd(B, H)), v.copy_(rnd(B, H)), q.copy_(rnd(B, H * G))
        add(k, v, table, lengths, np.arange(B + 1), np.array([[45 + x for x in lengths]]))
        lengths = [x + 1 for x in lengths]
        for gr, _ in graphs:                       # the second replay writes the same tokens again
            gr.replay()
        torch.cuda.synchronize()
        same_bytes(cache.pages.cpu().numpy(), shadow, f"step {i}")
        for _, (qr, full, win) in graphs:
            check_attend(full, qr, cache, signs, SCALE, table, lengths, prefix=(pre, 45))
            check_attend(win, qr, cache, signs, SCALE, table, lengths, window=16, sinks=2)
        assert torch.equal(graphs[0][1][1], graphs[1][1][1])
        start += 1
        after += 1
        pos += 1
    assert cache.status() == 0


def test_agrees_with_the_contiguous_cache():
    # the same tokens in both caches: the same codes, and outputs within the two kernels' roundings
    B, H, G, n = 2, 2, 4, 333
    g = torch.Generator(device="cuda").manual_seed(12)
    k, v = torch.randn((2, B, n, H, 128), generator=g, device="cuda", dtype=torch.bfloat16)
    q = torch.randn((B, H * G, 128), generator=g, device="cuda", dtype=torch.bfloat16)
    flat = kv.Cache(B, H, 384, seed=3)
    flat.append(k, v)
    cache, signs = new_cache(8, H, 128)
    table = np.array([[7, 1, 4], [0, 2, 5]], np.int32)
    cache.append(k.reshape(B * n, H, 128), v.reshape(B * n, H, 128), dev(table), dev([0, 0], torch.int32),
                 dev([0, n, 2 * n], torch.int32))
    a = flat.attend(q, SCALE).double().cpu().numpy()
    out = cache.attend(q, SCALE, dev(table), dev([n, n], torch.int32))
    check_attend(out, q, cache, signs, SCALE, table, [n, n])
    eps = torch.finfo(q.dtype).eps
    assert np.abs(ref.to_np(out) - a).max() <= (1e-3 + 3 * 2.0 ** -11 + eps / 2) * np.abs(a).max() * 4


def test_tables_that_are_views():
    # rows of a wider table, lengths and starts out of the middle of longer vectors
    lengths, page = [70, 33, 128], 32
    cache, signs, table, pre = filled(lengths, page, 2, 90, prefix=50)
    wide = torch.full((3, 11), -7, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + table.shape[1]] = dev(table)
    many = torch.full((8,), -1, dtype=torch.int32, device="cuda")
    many[3:6] = dev(lengths, torch.int32)
    q = torch.randn((3, 4, 128), device="cuda", dtype=torch.float16)
    tab, n = wide[:, 2:2 + table.shape[1]], many[3:6]
    check_attend(cache.attend(q, SCALE, tab, n), q, cache, signs, SCALE, table, lengths)
    out = cache.attend_shared(q, SCALE, dev(pre), dev([50], torch.int32), tab, n)
    check_attend(out, q, cache, signs, SCALE, table, lengths, prefix=(pre, 50))
    k = torch.randn((3, 2, 128), device="cuda", dtype=torch.float16)
    before = cache.pages.cpu().numpy()
    start = [x - 1 for x in lengths]
    many[3:6] = dev(start, torch.int32)
    cache.append(k, k, tab, many[3:6], dev([0, 1, 2, 3], torch.int32))
    same_bytes(cache.pages.cpu().numpy(), ref.append(before, ref.to_np(k), ref.to_np(k), table, start, [0, 1, 2, 3], signs))
    assert cache.status() == 0


def test_another_stream_and_default_results():
    lengths = [300, 40]
    cache, signs, table, _ = filled(lengths, 64, 2, 77)
    q = torch.randn((2, 4, 128), device="cuda", dtype=torch.float16)
    tab, n = dev(table), dev(lengths, torch.int32)
    torch.cuda.synchronize()
    first = cache.attend(q, SCALE, tab, n)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [cache.attend(q, SCALE, tab, n, stream=s) for s in streams for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(first, o) for o in outs)


def step_of(i, graphed):
    """A decode step of its own cache: append, attend and both forms of the shared attend; run(stream) -> results."""
    lengths, prefix, page = [150 + i, 1, 33, 64] * 6, 400, 64
    cache, _, table, pre = filled(lengths, page, 2, 120 + i, prefix=prefix)
    g = torch.Generator(device="cuda").manual_seed(i)
    q = torch.randn((24, 4, 128), generator=g, device="cuda", dtype=torch.bfloat16)
    k, v = torch.randn((2, 24, 2, 128), generator=g, device="cuda", dtype=torch.bfloat16)
    tab, n, plen = dev(table), dev(lengths, torch.int32), dev([prefix], torch.int32)
    cu = torch.arange(25, dtype=torch.int32, device="cuda")
    rope, at = kv.Rope(dev(rope_table(300, 128))), cu[:24]
    wide = torch.full((70000 * 128 // (page * 48 * 2),), -1, dtype=torch.int32, device="cuda")
    wide[:len(pre)] = dev(pre)
    start = n - 1

    def run(stream):
        turned = cache.append(k, v, tab, start, cu, rope, at, q=q, stream=stream)
        return [turned, cache.attend(turned, SCALE, tab, n, window=40, sinks=3, stream=stream)] + \
            [cache.attend_shared(turned, SCALE, pages, plen, tab, n, stream=stream) for pages in (dev_pre, wide)]

    dev_pre = dev(pre)
    torch.cuda.synchronize()
    if not graphed:
        return cache, run
    run(None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run(None)

    def replay(stream, inputs=run):  # the graph reads the tensors that `run` holds
        with torch.cuda.stream(stream):
            graph.replay()
            return [x.clone() for x in outs]

    return cache, replay


@pytest.mark.parametrize("graphed", [False, True])
def test_two_threads_at_once(graphed):
    # steps of two caches on two streams, launched by two host threads: as one after the other
    steps = [step_of(i, graphed) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in steps]
    alone = []
    for (_, run), s in zip(steps, streams):
        alone.append(run(s))
        torch.cuda.synchronize()
    with concurrent.futures.ThreadPoolExecutor(2) as pool:
        both = list(pool.map(lambda x: [x[0][1](x[1]) for _ in range(20)], zip(steps, streams)))
    torch.cuda.synchronize()
    for one, many in zip(alone, both):
        for outs in many:
            assert all(torch.equal(a, b) for a, b in zip(one, outs))
    assert all(cache.status() == 0 for cache, _ in steps)


def test_offsets_past_32_bits():
    # a buffer of more than 4 GiB: pages near its end
    H, page = 8, 4096
    num = (5 << 30) // (H * (page // 32) * 3200)
    cache, signs = new_cache(num, H, page)
    table = np.array([[num - 1, num - 2]], np.int32)
    n = 4200
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = torch.randn((2, n, H, 128), generator=g, device="cuda", dtype=torch.bfloat16)
    cache.append(k, v, dev(table), dev([0], torch.int32), dev([0, n], torch.int32))
    q = torch.randn((1, H, 128), generator=g, device="cuda", dtype=torch.bfloat16)
    out = cache.attend(q, SCALE, dev(table), dev([n], torch.int32))
    small = kv.PagedCache.wrap(cache.pages[-2:].contiguous(), cache.signs)
    near = np.array([[1, 0]], np.int32)
    check_attend(out, q, small, signs, SCALE, near, [n])
    assert cache.status() == 0


def test_refusals_of_the_binding():
    cache, _ = new_cache(4, 2, 64)
    q = torch.zeros((1, 4, 128), device="cuda", dtype=torch.float16)
    tab, n = dev([[0, 1]], torch.int32), dev([5], torch.int32)
    for bad in (lambda: cache.attend(q.cpu(), SCALE, tab, n), lambda: cache.attend(q, SCALE, tab.cpu(), n),
                lambda: cache.attend(q, SCALE, tab.long(), n), lambda: cache.attend(q, SCALE, tab, dev([5, 6], torch.int32)),
                lambda: cache.attend(q[:, :, :64], SCALE, tab, n), lambda: cache.attend(q, SCALE, tab, n, out=q.float()),
                lambda: cache.attend_shared(q, SCALE, tab[0, :0], n, tab, n),
                lambda: cache.attend_shared(q, SCALE, tab[0], tab[0], tab, n),
                lambda: kv.PagedCache.wrap(cache.pages[:, :, :, :100], cache.signs),
                lambda: kv.PagedCache.wrap(cache.pages, cache.signs[:1])):
        with pytest.raises(ValueError):
            bad()
    for args, code in (((q.float(), SCALE, tab, n), -2), ((q[:, :3].contiguous(), SCALE, tab, n), -1)):
        with pytest.raises(kv.Kv1bError) as e:
            cache.attend(*args)
        assert e.value.code == code
    with pytest.raises(kv.Kv1bError):
        cache.attend(q, SCALE, tab, n, window=-1)
    k = torch.zeros((3, 2, 128), device="cuda", dtype=torch.float16)
    ok = (tab, dev([0], torch.int32), dev([0, 3], torch.int32))
    for bad in (lambda: cache.append(k, k.float(), *ok), lambda: cache.append(k[:, :1], k[:, :1], *ok),
                lambda: cache.append(k, k, tab, dev([0, 1], torch.int32), ok[2]),
                lambda: cache.append(k, k, *ok, positions=n), lambda: cache.append(k, k, *ok, q_out=k),
                lambda: cache.append(k, k, *ok, q=k[:2]),
                lambda: cache.append(k, k, *ok, rope=kv.Rope(torch.zeros((4, 128), device="cuda"))),
                lambda: kv.Rope(torch.zeros((4, 12), device="cuda")), lambda: kv.Rope(torch.zeros((4, 128))),
                lambda: kv.Rope(torch.zeros((4, 128), device="cuda"), sections=[32, 16])):
        with pytest.raises(ValueError):
            bad()
    # nothing to do is no error
    assert cache.append(k[:0], k[:0], tab, dev([0], torch.int32), dev([0, 0], torch.int32)) is None
    assert cache.attend(q[:0], SCALE, tab[:0], n[:0]).shape == (0, 4, 128)
    assert cache.status() == 0
