"""Host checks of the kv1b_paged_* calls: what they refuse, with which code, before any launch; and the
plain CPU forms that the GPU tests compare with.  No kernel runs here."""
import ctypes

import numpy as np
import pytest

import oracle
import long_context_decode_kv1b_b200 as kv
import paged_reference as ref
from long_context_decode_kv1b_b200 import build, paged

P = 0x100000  # an address that no refused call looks at


@pytest.fixture(scope="module")
def lib():
    build.build()
    return kv.lib()


def desc(**kw):
    base = dict(pages=P, signs=P, d_status=0, num_pages=8, num_kv_heads=2, page_tokens=64, reserved=0)
    base.update(kw)
    return paged.PagedDesc(*(base[f] for f, _ in paged.PagedDesc._fields_))


def rope(**kw):
    base = dict(cos_sin=P, num_positions=16, rot_dim=128, axes=1, interleaved=0, sections=(ctypes.c_int32 * 3)(64, 0, 0),
                reserved=0)
    base.update(kw)
    return paged.RopeDesc(*(base[f] for f, _ in paged.RopeDesc._fields_))


def test_layouts():
    assert ctypes.sizeof(paged.PagedDesc) == 3 * 8 + 4 * 4
    assert ctypes.sizeof(paged.RopeDesc) == 8 + 4 * 4 + 3 * 4 + 4


def test_bytes(lib):
    assert lib.kv1b_paged_bytes(10, 8, 128, 64) == 10 * 8 * 2 * 3200
    assert lib.kv1b_paged_bytes(1 << 20, 8, 128, 4096) == (1 << 20) * 8 * 128 * 3200
    for bad in ((0, 8, 128, 64), (1, 0, 128, 64), (1, 1025, 128, 64), (1, 8, 64, 64), (1, 8, 128, 48), (1, 8, 128, 16),
                (1, 8, 128, 8192)):
        assert lib.kv1b_paged_bytes(*bad) == 0
    d = desc()
    assert lib.kv1b_paged_attend_workspace_bytes(ctypes.addressof(d), 8) > 0
    assert lib.kv1b_paged_shared_workspace_bytes(ctypes.addressof(d), 4, 8, 5) > 0
    for hq in (0, 3, 18):
        assert lib.kv1b_paged_attend_workspace_bytes(ctypes.addressof(d), hq) == 0
    assert lib.kv1b_paged_shared_workspace_bytes(ctypes.addressof(d), 0, 8, 5) == 0
    assert lib.kv1b_paged_shared_workspace_bytes(ctypes.addressof(d), 1025, 8, 5) == 0
    assert lib.kv1b_paged_shared_workspace_bytes(ctypes.addressof(d), 4, 8, 0) == 0


def test_signs_refusals(lib):
    assert lib.kv1b_paged_signs(None, 0, 1, P, None) == -1
    assert lib.kv1b_paged_signs(P, 0, 4, P, None) == -1
    assert lib.kv1b_paged_signs(P + 4, 0, 1, P, None) == -4


APPEND = dict(cache=None, k=P, v=P, dtype=1, num_tokens=4, kst=256, ksh=128, vst=256, vsh=128, seqs=2, cu=P, start=P, table=P,
              tstride=4, max_pages=4, rope=None, pos=None, pstride=0, q=None, qo=None, hq=0, qs0=0, qs1=0, os0=0, os1=0, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(k=None), -1), (dict(v=None), -1), (dict(cu=None), -1), (dict(start=None), -1), (dict(table=None), -1),
    (dict(dtype=3), -1), (dict(num_tokens=-1), -1), (dict(seqs=0), -1), (dict(seqs=1025, tstride=4), -2),
    (dict(max_pages=0), -1), (dict(tstride=3), -1), (dict(tstride=-4), -1), (dict(kst=-256), -1), (dict(vsh=-128), -1),
    (dict(k=P + 8), -4), (dict(ksh=130), -4), (dict(cu=P + 2), -4), (dict(num_tokens=(1 << 28) + 1), -2),
    (dict(max_pages=1 << 29, tstride=1 << 29), -2),
    (dict(q=P), -1), (dict(qo=P), -1), (dict(q=P, qo=P, hq=0), -1), (dict(q=P, qo=P, hq=1025), -1),
    (dict(q=P, qo=P, hq=8, qs0=1026, qs1=128, os0=1024, os1=128), -4), (dict(q=P + 4, qo=P, hq=8, os0=1024, os1=128), -4),
    (dict(q=P, qo=P, hq=8, qs0=1024, qs1=128, os0=0, os1=128), -1), (dict(q=P, qo=P, hq=8, qs0=1024, qs1=128, os0=1024, os1=64), -1),
    (dict(q=P, qo=P, hq=1000, num_tokens=1 << 27, os0=128000, os1=128), -2),
    (dict(rope=dict(), pos=None), -1), (dict(rope=dict(cos_sin=None), pos=P), -1), (dict(rope=dict(rot_dim=0), pos=P), -1),
    (dict(rope=dict(rot_dim=130), pos=P), -1), (dict(rope=dict(rot_dim=12, sections=(ctypes.c_int32 * 3)(6, 0, 0)), pos=P), -2),
    (dict(rope=dict(axes=4), pos=P), -1), (dict(rope=dict(axes=0), pos=P), -1),
    (dict(rope=dict(sections=(ctypes.c_int32 * 3)(60, 0, 0)), pos=P), -1),
    (dict(rope=dict(axes=2, sections=(ctypes.c_int32 * 3)(65, -1, 0)), pos=P, pstride=4), -1),
    (dict(rope=dict(axes=2, sections=(ctypes.c_int32 * 3)(32, 32, 0)), pos=P, pstride=3), -1),
    (dict(rope=dict(cos_sin=P + 8), pos=P), -4),
])
def test_append_refusals(lib, change, code):
    a = dict(APPEND, **{k: v for k, v in change.items() if k != "rope"})
    d, r = desc(), None
    a["cache"] = ctypes.addressof(d)
    if "rope" in change:
        r = rope(**change["rope"])
        a["rope"] = ctypes.addressof(r)
    assert lib.kv1b_paged_append(*a.values()) == code


@pytest.mark.parametrize("change", [dict(pages=None), dict(signs=None), dict(num_pages=0), dict(num_kv_heads=0),
                                    dict(num_kv_heads=1025), dict(page_tokens=48), dict(page_tokens=16), dict(pages=P + 64)])
def test_bad_descriptors(lib, change):
    d = desc(**change)
    at = ctypes.addressof(d)
    assert lib.kv1b_paged_append(*dict(APPEND, cache=at).values()) == -1
    assert lib.kv1b_paged_attend(at, P, 1, 8, 0.1, 2, P, 4, 4, P, 0, 0, P, P, 1 << 30, None) == -1
    assert lib.kv1b_paged_attend_shared(at, P, 1, 8, 0.1, 2, P, 4, P, P, 4, 4, P, P, P, 1 << 30, None) == -1


def test_nothing_to_append(lib):
    d = desc()
    assert lib.kv1b_paged_append(*dict(APPEND, cache=ctypes.addressof(d), num_tokens=0).values()) == 0


ATTEND = dict(q=P, dtype=1, hq=8, scale=0.1, seqs=2, table=P, tstride=4, max_pages=4, lengths=P, window=0, sinks=0, out=P, ws=P,
              wsb=1 << 30, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(q=None), -1), (dict(out=None), -1), (dict(ws=None), -1), (dict(table=None), -1), (dict(lengths=None), -1),
    (dict(dtype=0), -2), (dict(dtype=5), -1), (dict(hq=7), -1), (dict(hq=18), -2), (dict(seqs=0), -1), (dict(seqs=2000), -2),
    (dict(window=-1), -1), (dict(sinks=-1), -1), (dict(scale=float("nan")), -1), (dict(q=P + 8), -4), (dict(ws=P + 16), -4),
    (dict(wsb=64), -5), (dict(max_pages=1 << 29, tstride=1 << 29), -2), (dict(tstride=1), -1)])
def test_attend_refusals(lib, change, code):
    d = desc()
    a = dict(ATTEND, **change)
    assert lib.kv1b_paged_attend(ctypes.addressof(d), *a.values()) == code
    if not {"window", "sinks"} & set(change):
        args = [a[x] for x in ("q", "dtype", "hq", "scale", "seqs")] + [P, 4, P] + \
               [a[x] for x in ("table", "tstride", "max_pages", "lengths", "out", "ws", "wsb", "stream")]
        assert lib.kv1b_paged_attend_shared(ctypes.addressof(d), *args) == code


def test_shared_prefix_refusals(lib):
    d = desc()
    tail = (P, 4, 4, P, P, P, 1 << 30, None)
    for pre, code in (((None, 4, P), -1), ((P, 0, P), -1), ((P, 4, None), -1), ((P + 2, 4, P), -4), ((P, 1 << 30, P), -2)):
        assert lib.kv1b_paged_attend_shared(ctypes.addressof(d), P, 1, 8, 0.1, 2, *pre, *tail) == code


@pytest.mark.parametrize("change", [
    dict(qs0=1024, qs1=128, os0=128, os1=128), dict(qs0=1024, qs1=128, os0=1024, os1=256),       # rows over one another
    dict(q=P + 256, qs0=1024, qs1=128, os0=1024, os1=128), dict(q=P, qs0=2048, qs1=128, os0=1024, os1=128),
    dict(q=P + 64, qs0=1024, qs1=128, os0=1024, os1=128), dict(q=P, qs0=0, qs1=0, os0=1024, os1=128),
    dict(k=P + 2 * 1024, kst=2048, qs0=1024, qs1=128, q=2 * P, os0=1024, os1=128),
    dict(v=P + 2 * 896, vst=1024, qs0=1024, qs1=128, q=2 * P, os0=1024, os1=128)])
def test_append_refuses_rows_that_meet(lib, change):
    d = desc()
    a = dict(APPEND, cache=ctypes.addressof(d), k=3 * P, v=4 * P, q=P, qo=P, hq=8)
    a.update(change)
    assert lib.kv1b_paged_append(*a.values()) == -1


@pytest.mark.parametrize("out", [P + 128 * 2, P + 2 * 8 * 256 - 16, P - 16, P - 2 * 8 * 256 + 16])
def test_attend_refuses_results_over_a_part_of_the_queries(lib, out):
    d = desc()
    a = dict(ATTEND, out=out, ws=2 * P)
    assert lib.kv1b_paged_attend(ctypes.addressof(d), *a.values()) == -1
    args = [a[x] for x in ("q", "dtype", "hq", "scale", "seqs")] + [P, 4, P] + \
           [a[x] for x in ("table", "tstride", "max_pages", "lengths", "out", "ws", "wsb", "stream")]
    assert lib.kv1b_paged_attend_shared(ctypes.addressof(d), *args) == -1
    for clear in (P + 2 * 8 * 256, P - 2 * 8 * 256, P):  # these pass on to the workspace's check
        assert lib.kv1b_paged_attend(ctypes.addressof(d), *dict(ATTEND, out=clear, wsb=64).values()) == -5


def test_one_row_for_all(lib):
    # positions of a stride of 0 and, where it is only read, a page table of one: taken, up to the next check
    d, r = desc(), rope(axes=3, sections=(ctypes.c_int32 * 3)(32, 16, 16))
    at, ro = ctypes.addressof(d), ctypes.addressof(r)
    assert lib.kv1b_paged_append(*dict(APPEND, cache=at, rope=ro, pos=P, pstride=0, num_tokens=0).values()) == 0
    assert lib.kv1b_paged_append(*dict(APPEND, cache=at, rope=ro, pos=P, pstride=0, q=P).values()) == -1
    assert lib.kv1b_paged_append(*dict(APPEND, cache=at, rope=ro, pos=P + 2, pstride=0).values()) == -4
    assert lib.kv1b_paged_append(*dict(APPEND, cache=at, tstride=0).values()) == -1  # two sequences in one page
    assert lib.kv1b_paged_attend(at, *dict(ATTEND, tstride=0, wsb=64).values()) == -5
    assert lib.kv1b_paged_attend_shared(at, P, 1, 8, 0.1, 2, P, 4, P, P, 0, 4, P, P, P, 64, None) == -5


# ---- the plain forms themselves
def test_reference_turn_is_a_rotation_by_the_positions_angle():
    rng = np.random.default_rng(0)
    half = 16
    ang = rng.uniform(-3, 3, (7, half))
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    x = rng.standard_normal((2, 128)).astype(np.float32)
    for inter in (False, True):
        y = ref.turn(x, cs, [3, 5], [10, 6], inter)
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
            th = ang[3 if i < 10 else 5, i]
            z = (x[:, a].astype(np.complex128) + 1j * x[:, b]) * np.exp(1j * th)
            # two products and a sum, cos and sin rounded once
            assert np.abs(y[:, a] + 1j * y[:, b] - z).max() <= 4 * 2.0 ** -24 * np.abs(z).max() * 2
        assert np.array_equal(y[:, 2 * half:], x[:, 2 * half:])


def test_reference_block_fields_round_trip():
    rng = np.random.default_rng(1)
    signs = oracle.signs(3)
    pages = rng.integers(0, 256, (3, 2, 2, ref.BYTES), dtype=np.uint8)
    k, v = rng.standard_normal((2, 40, 2, 128)).astype(np.float32)
    got = ref.append(pages, k, v, [[2, 0]], [30], [0, 40], signs)
    assert np.array_equal(got[1], pages[1])
    for h in range(2):
        e = oracle.encode(k[:, h], v[:, h], signs)
        sign, val, nc, _, _ = part = ref.gather(got, [2, 0], h, np.arange(30, 70))
        bits = ((e["bits"][:, :, None] >> np.arange(32, dtype=np.uint32)) & 1).reshape(40, 128)
        assert np.array_equal(sign > 0, bits > 0)
        assert np.array_equal(val, oracle.dequant(e["codes"], e["sm"]))
        assert np.array_equal(nc, (e["norm"] * e["cinv"]).astype(np.float64))
        q = rng.standard_normal(128).astype(np.float32)
        out = ref.Row(q, signs, 0.1, [part]).out
        assert np.abs(out - oracle.attend(e, q, signs, 0.1)).max() < 1e-5
