"""Refusals of the paged-cache entry points (checked before anything is
launched, so on the CPU with addresses that are never read) and the host-made
rotary table.  No GPU needed."""
import ctypes
import math

import numpy as np
import pytest

import oracle
from tile_level_overlap_gb300 import build, mk

ADDR = 1 << 20  # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    build.build()
    return mk.lib()


def cache(**kw):
    f = dict(k=ADDR, v=ADDR, workspace=ADDR, status=None, page_stride=16 * 8 * 128, head_stride=16 * 128,
             token_stride=128, n_q_heads=32, n_kv_heads=8, head_dim=128, page_size=16, n_pages=100,
             dtype=mk.MK_BF16)
    f.update(kw)
    return mk.mk_paged_cache(*[f[n] for n, _ in mk.mk_paged_cache._fields_])


def batch(**kw):
    f = dict(block_table=ADDR, cu_new=ADDR, kv_lens=ADDR, positions=ADDR, slots=ADDR, n=4, max_blocks=8,
             max_tokens=0, max_new=1, page_size=16)
    f.update(kw)
    return mk.mk_paged_batch(*[f[n] for n, _ in mk.mk_paged_batch._fields_])


def attention(lib, c, b, q=ADDR, qs=4096, out=2 * ADDR, os=4096, lse=None, scale=0.0, window=0):
    return lib.mk_paged_attention(ctypes.byref(c) if c else None, ctypes.byref(b) if b else None, q, qs,
                                  out, os, lse, scale, window, None)


BAD_CACHE = [
    (dict(k=None), 1), (dict(v=None), 1), (dict(k=ADDR + 8), 1), (dict(v=ADDR + 2), 1),
    (dict(status=ADDR + 1), 1), (dict(n_q_heads=0), 1), (dict(n_kv_heads=0), 1), (dict(n_pages=0), 1),
    (dict(dtype=2), 1), (dict(dtype=-1), 1), (dict(page_stride=100), 1), (dict(head_stride=-8), 1),
    (dict(token_stride=4), 1), (dict(token_stride=64), 1), (dict(head_dim=96), 5), (dict(head_dim=0), 5),
    (dict(page_size=8), 5), (dict(page_size=48), 5), (dict(page_size=512), 5),
    (dict(n_pages=1 << 27, page_size=16), 5),
]


@pytest.mark.parametrize("kw,code", BAD_CACHE)
def test_bad_caches_are_refused(lib, kw, code):
    b = batch(page_size=kw.get("page_size", 16)) if kw.get("page_size", 16) in (16, 32) else batch()
    assert attention(lib, cache(**kw), b) == code
    args = (ADDR, 4096, ADDR, 1024, ADDR, 1024, ADDR, 4096, None, None, 1e-6, None, None, 0, ADDR, 0, None)
    assert lib.mk_paged_append(ctypes.byref(cache(**kw)), *args) == code


@pytest.mark.parametrize("kw,code", [
    (dict(block_table=None), 1), (dict(cu_new=None), 1), (dict(kv_lens=None), 1), (dict(cu_new=ADDR + 2), 1),
    (dict(n=0), 1), (dict(n=mk.MK_PAGED_MAX_REQUESTS + 1), 5), (dict(max_blocks=0), 1),
    (dict(max_tokens=-1), 1), (dict(max_new=0), 1), (dict(page_size=32), 1), (dict(page_size=17), 5),
    (dict(n=4096, max_blocks=1 << 20), 5), (dict(n=1, max_blocks=1 << 27), 5), (dict(n=1, max_blocks=(1 << 26) + 1), 5),
    (dict(n=4, max_blocks=1 << 26, max_tokens=400), 5),
])
def test_bad_batches_are_refused(lib, kw, code):
    assert attention(lib, cache(), batch(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(out=ADDR), 1), (dict(q=ADDR + 4), 1), (dict(out=ADDR + 8), 1),
    (dict(qs=4000), 1), (dict(os=4090), 1), (dict(qs=4100), 1), (dict(qs=1 << 38), 1), (dict(lse=ADDR + 2), 1), (dict(window=-1), 1),
    (dict(scale=math.nan), 1), (dict(scale=math.inf), 1),
])
def test_bad_attention_arguments_are_refused(lib, kw, code):
    assert attention(lib, cache(), batch(), **kw) == code


def test_attention_refusals_of_whole_structs(lib):
    assert attention(lib, None, batch()) == 1
    assert attention(lib, cache(), None) == 1
    assert attention(lib, cache(workspace=None), batch()) == 1
    assert attention(lib, cache(workspace=ADDR + 8), batch()) == 1
    assert attention(lib, cache(n_q_heads=33), batch(), qs=4224, os=4224) == 1
    assert attention(lib, cache(n_q_heads=65, n_kv_heads=1), batch(), qs=8320, os=8320) == 5
    # no rows: nothing to do, nothing launched
    assert attention(lib, cache(), batch()) == 0


@pytest.mark.parametrize("hq,hkv,rows,width", [
    (65537, 65537, 1, 8), (1 << 23, 1, 700, 8), (1 << 24, 1 << 20, 1, 8), (0x7fffffff, 0x7fffffff, 1, 8),
    # 2^31 rows on 2^16 heads over 2^30 keys: work whose count passes 64 bits
    (1 << 16, 1 << 16, 0x7fffffff, 1 << 26), (1 << 16, 1 << 14, 1 << 30, 1 << 26),
])
def test_sizes_past_the_counters_are_refused(lib, hq, hkv, rows, width):
    c = cache(n_q_heads=hq, n_kv_heads=hkv)
    b = batch(n=1, max_blocks=width, max_tokens=rows)
    assert attention(lib, c, b, qs=hq * 128 + 8, os=hq * 128 + 8) == 5
    if hq > mk.MK_PAGED_MAX_HEADS:
        args = (ADDR, hq * 128, ADDR, hkv * 128, ADDR, hkv * 128, ADDR, hq * 128, None, None, 1e-6, None, None, 0,
                ADDR, rows, None)
        assert lib.mk_paged_append(ctypes.byref(c), *args) == 5


def test_bad_append_arguments_are_refused(lib):
    rope = mk.mk_rope()
    assert lib.mk_rope_init(ctypes.byref(rope), 128, 1e4, None, 1, None) == 0
    ok = dict(q=ADDR, qs=4096, k=ADDR, ks=1024, v=ADDR, vs=1024, qo=ADDR, qos=4096, qn=None, kn=None, eps=1e-6,
              rope=ctypes.byref(rope), pos=ADDR, ps=0, slots=ADDR, n=0)

    def call(c=None, **kw):
        return lib.mk_paged_append(ctypes.byref(c or cache()), *{**ok, **kw}.values(), None)

    assert call() == 0
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(qo=None), dict(slots=None), dict(slots=ADDR + 2),
               dict(q=ADDR + 8), dict(qn=ADDR + 2), dict(kn=ADDR + 8), dict(qs=4092), dict(qs=4088), dict(ks=1016),
               dict(vs=1028), dict(qos=0), dict(eps=-1.0), dict(eps=math.nan), dict(n=-1), dict(pos=None),
               dict(pos=ADDR + 1), dict(ps=-1), dict(qos=4104)):
        assert call(**kw) == 1, kw
    assert call(qo=2 * ADDR, qos=4104) == 0
    assert call(rope=None, pos=None) == 0
    # a rotation wider than the head
    assert call(cache(head_dim=64), qs=4096) == 1
    bad = mk.mk_rope.from_buffer_copy(rope)
    bad.axis[3] = 1
    assert call(rope=ctypes.byref(bad)) == 1
    bad = mk.mk_rope.from_buffer_copy(rope)
    bad.rotary_dim = 24
    assert call(rope=ctypes.byref(bad)) == 1


def test_bad_table_arguments_are_refused(lib):
    ok = dict(ctx=ADDR, new=ADDR, free=ADDR, cap=10, n_free=ADDR, n_left=ADDR + 4, status=None)

    def call(b=None, **kw):
        return lib.mk_paged_tables(ctypes.byref(b or batch()), *{**ok, **kw}.values(), None)

    for kw in (dict(ctx=None), dict(new=None), dict(free=None), dict(cap=-1), dict(n_free=None), dict(n_left=None),
               dict(n_left=ADDR), dict(ctx=ADDR + 1), dict(status=ADDR + 2), dict(n_left=ADDR + 5)):
        assert call(**kw) == 1, kw
    assert call(batch(max_tokens=3, positions=None)) == 1
    assert call(batch(max_tokens=3, slots=None)) == 1
    assert call(batch(max_tokens=3, slots=ADDR + 2)) == 1
    assert call(batch(n=0)) == 1
    assert call(batch(n=5000)) == 5
    assert lib.mk_paged_tables(None, *ok.values(), None) == 1


@pytest.mark.parametrize("batch_kw,call_kw", [
    (dict(), dict(ctx=12 * ADDR)),                       # the batch's own kv_lens as the cached lengths
    (dict(), dict(ctx=12 * ADDR + 12)),                  # one word in common
    (dict(), dict(new=12 * ADDR - 12)), (dict(), dict(new=11 * ADDR + 16)), (dict(), dict(free=10 * ADDR + 124)),
    (dict(), dict(free=14 * ADDR - 36)), (dict(), dict(n_left=5 * ADDR)), (dict(), dict(n_left=4 * ADDR + 36)),
    (dict(), dict(n_left=2 * ADDR + 12)), (dict(), dict(status=5 * ADDR)), (dict(), dict(status=6 * ADDR)),
    (dict(slots=13 * ADDR), dict()), (dict(slots=13 * ADDR + 2396), dict()), (dict(cu_new=12 * ADDR - 16), dict()),
])
def test_tables_that_overlap_are_refused(lib, batch_kw, call_kw):
    # (free_pages at 14 * ADDR - 36 meets the slots with its last word)
    b = batch(**{**dict(block_table=10 * ADDR, cu_new=11 * ADDR, kv_lens=12 * ADDR, positions=13 * ADDR,
                        slots=14 * ADDR, max_tokens=600), **batch_kw})
    ok = dict(ctx=2 * ADDR, new=3 * ADDR, free=4 * ADDR, cap=10, n_free=5 * ADDR, n_left=6 * ADDR, status=None)
    assert lib.mk_paged_tables(ctypes.byref(b), *{**ok, **call_kw}.values(), None) == 1


@pytest.mark.parametrize("rot,theta,axes", [(16, 1e4, 1), (64, 5e5, 1), (128, 1e6, 3), (96, 1e4, 4)])
def test_rope_table_is_the_fraction_of_a_turn(lib, rot, theta, axes):
    half = rot // 2
    of = (ctypes.c_uint8 * half)(*[i % axes for i in range(half)])
    r = mk.mk_rope()
    assert lib.mk_rope_init(ctypes.byref(r), rot, theta, None, axes, of if axes > 1 else None) == 0
    assert (r.rotary_dim, r.n_axes) == (rot, axes)
    for i in range(half):
        want = theta ** (-2 * i / rot) / (2 * math.pi)
        # a few roundings of 2^-53 in pow, the division and the table
        assert abs(r.turn[i] / 2 ** 64 - want) <= 8 * 2 ** -53 * want + 2 ** -63
        assert r.axis[i] == (i % axes if axes > 1 else 0)


def test_rope_table_of_given_frequencies(lib):
    half = 8
    freq = [0.5, -0.25, 7.0, 0.0, -1e-20, 1e-9, 2 * math.pi, 100.0]
    r = mk.mk_rope()
    assert lib.mk_rope_init(ctypes.byref(r), 16, 0.0, (ctypes.c_double * half)(*freq), 1, None) == 0
    for i, f in enumerate(freq):
        got = r.turn[i] / 2 ** 64 * 2 * math.pi
        assert abs(math.remainder(got - f, 2 * math.pi)) <= 1e-13, (i, f)


def test_bad_rope_tables_are_refused(lib):
    r = mk.mk_rope()
    p = ctypes.byref(r)
    two = (ctypes.c_uint8 * 64)(*([0, 1] * 32))
    nan = (ctypes.c_double * 64)(*([math.nan] * 64))
    for args in ((None, 64, 1e4, None, 1, None), (p, 0, 1e4, None, 1, None), (p, 24, 1e4, None, 1, None),
                 (p, 144, 1e4, None, 1, None), (p, 64, 0.0, None, 1, None), (p, 64, -1.0, None, 1, None),
                 (p, 64, math.inf, None, 1, None), (p, 64, 1e4, None, 0, None), (p, 64, 1e4, None, 5, two),
                 (p, 64, 1e4, None, 2, None), (p, 64, 1e4, None, 1, two), (p, 64, 1e4, nan, 1, None)):
        assert lib.mk_rope_init(*args) == 1


def test_rope_sections_name_the_axes():
    r = mk.Rope(128, sections=[16, 24, 24])
    assert list(r.c.axis) == [0] * 16 + [1] * 24 + [2] * 24 and r.n_axes == 3
    r = mk.Rope(128, sections=[24, 20, 20], interleaved=True)
    assert list(r.c.axis) == [0, 1, 2] * 20 + [0] * 4
    with pytest.raises(ValueError):
        mk.Rope(128, sections=[16, 24])
    with pytest.raises(ValueError):
        mk.Rope(64, rotary_dim=128)


# ---- pins of the oracle these operators are tested against

def test_oracle_tables_hand_case():
    table = np.full((3, 4), -1)
    table[0, 0] = 9
    t = oracle.paged_tables([3, 0, 4], [2, 5, 0], [5, 6, 7, 8], 4, table, 4, 8)
    assert t["table"].tolist() == [[9, 8, -1, -1], [7, 6, -1, -1], [-1, -1, -1, -1]]
    assert t["cu_new"].tolist() == [0, 2, 7, 7] and t["kv_lens"].tolist() == [5, 5, 4]
    assert t["positions"].tolist() == [3, 4, 0, 1, 2, 3, 4, 0]
    assert t["slots"].tolist() == [39, 32, 28, 29, 30, 31, 24, -1]
    assert t["n_left"] == 1 and not t["refused"]


def test_oracle_attention_closed_forms():
    rng = np.random.default_rng(0)
    k, v = rng.standard_normal((3, 1, 4, 8)), rng.standard_normal((3, 1, 4, 8))
    table, q = np.array([[2, 0]]), rng.standard_normal((2, 1, 8))
    # one visible key: its value; q = 0: the mean; no key: zero
    out, lse, *_ = oracle.paged_attention(q, k, v, table, [0, 2], [5], 0.3, window=1)
    assert np.allclose(out[0, 0], v[2, 0, 3]) and np.allclose(out[1, 0], v[0, 0, 0])
    assert np.allclose(lse[1, 0], 0.3 * q[1, 0] @ k[0, 0, 0])
    out, lse, *_ = oracle.paged_attention(0 * q, k, v, table, [0, 2], [5], 0.3)
    assert np.allclose(out[0, 0], v[2, 0].mean(0)) and np.allclose(lse[:, 0], np.log([4, 5]))
    out, lse, *_ = oracle.paged_attention(q, k, v, table, [0, 2], [1], 0.3)
    assert (out[0] == 0).all() and lse[0, 0] == -np.inf and np.allclose(out[1, 0], v[2, 0, 0])


def test_oracle_rope_is_the_model_oracles():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 2, 64))
    pos = np.array([0, 1, 7, 100, 4096])
    inv = [1e4 ** (-2 * i / 64) for i in range(32)]
    got = oracle.rope_rows(x, [pos], [0] * 32, inv)
    z = x[..., :32] + 1j * x[..., 32:]
    z = z * np.exp(1j * pos[:, None] * np.array(inv))[:, None]
    assert np.allclose(got, np.concatenate([z.real, z.imag], -1))
