"""Pins of the float64 references of prompt attention and the 4-bit cache, and the host-side
checks of their entry points (no device needed)."""
from __future__ import annotations

import ctypes as C
import math

import numpy as np
import pytest

from oracle import prompt_int4_oracle as P


def test_prompt_attend_by_hand():
    # two positions, D = 4 (scale 1/2): scores of row 1 are 0 and ln 3, so p = (1/4, 3/4)
    q = np.zeros((2, 1, 4))
    q[1, 0, 0] = 2 * math.log(3.0)
    k = np.zeros((2, 1, 4))
    k[1, 0, 0] = 1.0
    v = np.zeros((2, 1, 4))
    v[0, 0], v[1, 0] = [4, 0, 0, 8], [0, 4, 0, 8]
    out, lse, _, _ = P.prompt_attend(q, k, v)
    np.testing.assert_allclose(out[:, 0], [[4, 0, 0, 8], [1, 3, 0, 8]], rtol=1e-14)
    np.testing.assert_allclose(lse[:, 0], [0.0, math.log(4.0)], rtol=1e-14, atol=1e-15)
    np.testing.assert_allclose(P.prompt_mass(q, k, lse)[:, 0], [1.25, 0.75], rtol=1e-14)


def test_prompt_mass_sums_to_rows_and_heads():
    r = np.random.default_rng(1)
    q, k, v = r.standard_normal((23, 6, 8)), r.standard_normal((23, 2, 8)), r.standard_normal((23, 2, 8))
    _, lse, _, _ = P.prompt_attend(q, k, v)
    np.testing.assert_allclose(P.prompt_mass(q, k, lse).sum(0), [23 * 3, 23 * 3], rtol=1e-12)


def test_int4_groups_by_hand():
    x = np.full((1, 64), 2.0)
    x[0, :32] = np.arange(32) % 16                       # 0..15: s = 1, z = 0, codes as they are
    c, s, z = P.int4_quantize(x)
    assert c[0, :32].tolist() == [i % 16 for i in range(32)] and (s[0, 0], z[0, 0]) == (1.0, 0.0)
    assert not c[0, 32:].any() and (s[0, 1], z[0, 1]) == (0.0, 2.0)      # constant group
    np.testing.assert_array_equal(P.int4_values(c, s, z), x)
    y = np.zeros(32)
    y[:4] = [0.0, 15.0, 0.5, 1.5]                        # ties go to the even code
    assert P.int4_quantize(y)[0][:4].tolist() == [0, 15, 0, 2]


@pytest.mark.parametrize("D", [64, 128])
def test_int4_page_keeps_every_nibble(D):
    r = np.random.default_rng(2)
    k, v = r.standard_normal((16, D)), r.standard_normal((16, D))
    page = P.int4_page(k, v)
    assert page.size == 20 * D
    # every code and half occurs once: sums over the page equal those over the entries
    for base, x in ((0, k), (8 * D, v)):
        b = page[base:base + 8 * D]
        assert int((b & 15).sum() + (b >> 4).sum()) == int(P.int4_quantize(x)[0].sum())
    halves = page[16 * D:].view(np.float16)
    for n, x in enumerate((P.int4_quantize(k)[1], P.int4_quantize(k)[2], P.int4_quantize(v)[1], P.int4_quantize(v)[2])):
        assert sorted(halves[n * D // 2:(n + 1) * D // 2].tolist()) == sorted(x.ravel().tolist())
    # the documented places of single elements
    c = P.int4_quantize(v)[0]
    i, g, rr, j = 11, D // 32 - 1, 5, 3
    byte = page[8 * D + i * D // 2 + (rr * (D // 32) + g) * 2 + 1]
    assert byte >> 4 == c[i, 32 * g + 4 * rr + j]


def test_int4_attend_is_softmax_attention():
    q, k = np.zeros((2, 4)), np.zeros((3, 4))
    v = np.eye(3, 4)
    k[:, 0] = [0.0, math.log(2.0), math.log(5.0)]
    q[1, 0] = 2.0
    out, p = P.int4_attend(q, k, v)
    np.testing.assert_allclose(p[:, 0], [1 / 3] * 3)
    np.testing.assert_allclose(p[:, 1], [1 / 8, 2 / 8, 5 / 8])
    np.testing.assert_allclose(out[1], [1 / 8, 2 / 8, 5 / 8, 0])
    assert P.int4_attend(q, k[:0], v[:0])[0].tolist() == [[0.0] * 4] * 2


def test_int4_evict_order():
    nan = float("nan")
    m = [5.0, 1.0, 1.0, nan, 0.0, 9.0, -1.0, 1.0]
    pos = [0, 1, 2, 4, 7, 8, 9, 10]
    assert P.int4_evict(m, pos, 11, 4, 1).tolist() == [0, 1, 5, 7]          # 7 is the newest
    assert P.int4_evict(m, pos, 11, 4, 0).tolist() == [0, 1, 2, 5]          # ties: the lower entries
    assert P.int4_evict(m, pos, 11, 7, 0).tolist() == [0, 1, 2, 4, 5, 6, 7]  # NaN goes first
    assert P.int4_evict(m, pos, 11, 8, 0).tolist() == list(range(8))
    assert P.int4_evict(m, pos, 11, 2, 11).tolist() == [0, 1]               # more newest ones than places


@pytest.fixture(scope="module")
def L():
    from kv_cache_eviction_gqa_b200 import binding as B
    from kv_cache_eviction_gqa_b200 import build
    build.build()
    return B.lib()


FAKE = 1 << 40          # a stand-in device address, never read


def _cache(**kw):
    from kv_cache_eviction_gqa_b200 import binding as B
    f = dict(B=2, Hkv=2, D=128, max_pages=4, n_pages=16, pages=FAKE, page_table=FAKE, lengths=FAKE, seen=FAKE,
             mass=FAKE, pos=FAKE, status=FAKE)
    f.update(kw)
    return B.QeInt4Cache(**f)


@pytest.mark.parametrize("bad,code", [
    (dict(Hq=7), -1), (dict(B=0), -1), (dict(T=-1), -1), (dict(dtype=2), -1), (dict(D=96), -2), (dict(Hq=18), -2),
    (dict(T=(1 << 30) + 1), -2), (dict(q=FAKE + 8), -1), (dict(qs=8 * 128 + 4), -1), (dict(qs=8 * 128 - 8), -1),
    (dict(ks=100), -1), (dict(cu=None), -1), (dict(status=None), -1), (dict(out=None), -1), (dict(out=FAKE + 2), -1)])
def test_prompt_refusals(L, bad, code):
    a = dict(q=FAKE, k=FAKE, v=FAKE, qs=8 * 128, ks=256, vs=256, cu=FAKE, B=2, T=64, Hq=8, Hkv=2, D=128, dtype=1,
             out=FAKE, lse=FAKE, status=FAKE)
    a.update(bad)
    assert L.qe_prompt_attend(a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["cu"], a["B"], a["T"], a["Hq"],
                              a["Hkv"], a["D"], a["dtype"], a["out"], a["lse"], a["status"], None) == code
    if "out" not in bad:
        assert L.qe_prompt_mass(a["q"], a["k"], a["qs"], a["ks"], a["lse"], a["cu"], a["B"], a["T"], a["Hq"], a["Hkv"],
                                a["D"], a["dtype"], FAKE, a["status"], None) == code


def test_prompt_of_no_rows_does_nothing(L):
    assert L.qe_prompt_attend(None, None, None, 0, 0, 0, FAKE, 1, 0, 8, 2, 128, 1, None, None, FAKE, None) == 0
    assert L.qe_prompt_mass(None, None, 0, 0, None, FAKE, 1, 0, 8, 2, 128, 1, None, FAKE, None) == 0


@pytest.mark.parametrize("bad,code", [
    (dict(D=96), -2), (dict(B=0), -1), (dict(max_pages=0), -1), (dict(n_pages=0), -1), (dict(pages=None), -1),
    (dict(pages=FAKE + 4), -1), (dict(status=None), -1), (dict(seen=None), -1), (dict(max_pages=1 << 26), -2)])
def test_int4_cache_refusals(L, bad, code):
    c, other = _cache(**bad), _cache(pages=2 * FAKE, lengths=2 * FAKE, seen=2 * FAKE, mass=2 * FAKE, pos=2 * FAKE)
    r = C.byref
    assert L.qe_int4_append(r(c), FAKE, FAKE, 256, 256, FAKE, 4, 1, None, None) == code
    assert L.qe_int4_read(r(c), FAKE, 4, None, 1, FAKE, FAKE, None) == code
    assert L.qe_int4_attend(r(c), FAKE, 1024, 8, 1, 1, FAKE, FAKE, 1 << 40, None) == code
    assert L.qe_int4_evict(r(c), r(other), 8, 0, None) == code
    assert L.qe_int4_evict(r(other), r(c), 8, 0, None) == code


def test_int4_call_refusals(L):
    r = C.byref
    c, d = _cache(), _cache(pages=2 * FAKE, lengths=2 * FAKE, seen=2 * FAKE, mass=2 * FAKE, pos=2 * FAKE)
    assert L.qe_int4_append(None, FAKE, FAKE, 256, 256, FAKE, 4, 1, None, None) == -1
    for args in ((None, FAKE, 256, 256, FAKE, 4, 1), (FAKE, FAKE, 254, 256, FAKE, 4, 1), (FAKE, FAKE, 258, 256, FAKE, 4, 1),
                 (FAKE + 4, FAKE, 256, 256, FAKE, 4, 1), (FAKE, FAKE, 256, 256, None, 4, 1), (FAKE, FAKE, 256, 256, FAKE, -1, 1),
                 (FAKE, FAKE, 256, 256, FAKE, 4, 2)):
        assert L.qe_int4_append(r(c), *args, None, None) == -1
    assert L.qe_int4_append(r(c), None, None, 0, 0, FAKE, 0, 1, None, None) == 0
    assert L.qe_int4_read(r(c), FAKE, 4, None, 1, None, FAKE, None) == -1
    assert L.qe_int4_read(r(c), FAKE, 0, None, 1, None, None, None) == 0
    n = L.qe_int4_scratch_bytes(2, 8, 2, 128, 4)
    assert n >= 4 * 64 * 4 * 4                      # every entry's scores
    assert L.qe_int4_scratch_bytes(2, 7, 2, 128, 4) == 0 and L.qe_int4_scratch_bytes(2, 18, 2, 128, 4) == 0
    assert L.qe_int4_scratch_bytes(2, 8, 2, 96, 4) == 0 and L.qe_int4_scratch_bytes(2, 8, 2, 128, 1 << 26) == 0
    assert L.qe_int4_attend(r(c), FAKE, 1024, 8, 1, 1, FAKE, FAKE, n - 1, None) == -8
    assert L.qe_int4_attend(r(c), FAKE, 1024, 7, 1, 1, FAKE, FAKE, n, None) == -1
    assert L.qe_int4_attend(r(c), FAKE, 2304, 18, 1, 1, FAKE, FAKE, 1 << 40, None) == -2
    assert L.qe_int4_attend(r(c), FAKE, 1028, 8, 1, 1, FAKE, FAKE, n, None) == -1
    assert L.qe_int4_attend(r(c), FAKE, 1024, 8, 1, 1, FAKE, FAKE + 16, n, None) == -1
    big = _cache(B=40000)
    assert L.qe_int4_attend(r(big), FAKE, 1024, 8, 1, 1, FAKE, FAKE, 1 << 40, None) == -2
    for budget, recent in ((0, 0), (65, 0), (8, -1), (0x7fffffff, 0)):
        assert L.qe_int4_evict(r(c), r(d), budget, recent, None) == -1
    assert L.qe_int4_evict(r(c), r(c), 8, 0, None) == -1
    assert L.qe_int4_evict(r(c), r(_cache(pages=2 * FAKE, lengths=2 * FAKE, mass=2 * FAKE, pos=2 * FAKE)), 8, 0, None) == -1
    assert L.qe_int4_evict(r(c), r(_cache(D=64, pages=2 * FAKE)), 8, 0, None) == -1


def test_int4_evict_refuses_more_newest_than_the_budget(L):
    """Which of the newest entries to drop is not defined."""
    c, d = _cache(), _cache(pages=2 * FAKE, lengths=2 * FAKE, seen=2 * FAKE, mass=2 * FAKE, pos=2 * FAKE)
    assert L.qe_int4_evict(C.byref(c), C.byref(d), 8, 9, None) == -1


def test_a_stream_of_another_device_is_refused():
    from types import SimpleNamespace

    from kv_cache_eviction_gqa_b200 import binding
    with pytest.raises(ValueError, match="cuda:1"):
        binding._on(0, SimpleNamespace(device_index=1))
