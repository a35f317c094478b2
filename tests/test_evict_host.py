"""Host side of the bounded cache (no GPU): truncate and unshare of the
allocator, and the refusals of the C entry points before any device work."""
import ctypes

import pytest

import pagedattention_decode_gb300 as P
from pagedattention_decode_gb300 import _native


def test_truncate_releases_blocks_in_table_order():
    a = P.BlockAllocator(8, 16)
    s = a.create_sequence()
    a.append_tokens([s], [100])
    table = a.block_table(s)
    assert len(table) == 7 and a.num_free == 1
    a.truncate(s, 33)
    assert a.seq_len(s) == 33 and a.block_table(s) == table[:3] and a.num_free == 5
    # LIFO: the last block released is the next one taken
    t = a.create_sequence()
    slots, _ = a.append_tokens([t], [16])
    assert slots[0] // 16 == table[6]
    # the tail goes on where the cut left it
    slots, pairs = a.append_tokens([s], [1])
    assert slots == [table[2] * 16 + 1] and pairs == []
    a.truncate(s, 34)  # its own length: nothing happens
    assert a.seq_len(s) == 34 and len(a.block_table(s)) == 3
    a.truncate(s, 0)
    assert a.seq_len(s) == 0 and a.block_table(s) == []


def test_truncate_keeps_shared_blocks_alive():
    a = P.BlockAllocator(6, 4)
    s = a.create_sequence()
    a.append_tokens([s], [10])
    f = a.fork(s)
    table = a.block_table(s)
    a.truncate(s, 4)
    assert [a.refcount(b) for b in table] == [2, 1, 1] and a.block_table(f) == table and a.num_free == 3


def test_truncate_refusals():
    a = P.BlockAllocator(4, 4)
    s = a.create_sequence()
    a.append_tokens([s], [5])
    for n in (6, -1):
        with pytest.raises(P.PkvError) as e:
            a.truncate(s, n)
        assert e.value.status == 1
    with pytest.raises(P.PkvError) as e:
        a.truncate(99, 0)
    assert e.value.status == 4
    assert a.seq_len(s) == 5
    a.free_sequence(s)
    with pytest.raises(P.PkvError):
        a.truncate(s, 0)


def test_unshare_gives_private_blocks():
    a = P.BlockAllocator(12, 4)
    s = a.create_sequence()
    a.append_tokens([s], [10])
    f, g = a.fork(s), a.fork(s)
    old = a.block_table(s)
    # s and f leave the blocks; g, not listed, keeps them
    pairs = a.unshare([s, f])
    assert len(pairs) == 6 and [p[0] for p in pairs] == old + old and len({p[1] for p in pairs}) == 6
    assert a.block_table(s) == [p[1] for p in pairs[:3]] and a.block_table(f) == [p[1] for p in pairs[3:]]
    assert a.block_table(g) == old
    for x in (s, f, g):
        assert all(a.refcount(b) == 1 for b in a.block_table(x))
    assert a.unshare([s, f, g]) == []
    assert a.counters()["cow_copies"] == 6


def test_unshare_last_holder_keeps_the_block():
    a = P.BlockAllocator(6, 4)
    s = a.create_sequence()
    a.append_tokens([s], [8])
    f = a.fork(s)
    old = a.block_table(s)
    pairs = a.unshare([s, f])
    assert [p[0] for p in pairs] == old and a.block_table(f) == old


def test_unshare_leaves_the_prefix_trie_its_blocks():
    a = P.BlockAllocator(8, 4)
    toks = list(range(8))
    s = a.create_sequence()
    a.append_tokens([s], [8])
    old = a.block_table(s)
    a.prefix_insert(toks, old)
    pairs = a.unshare([s])
    assert [p[0] for p in pairs] == old and a.prefix_match(toks) == old and a.refcount(old[0]) == 1


def test_unshare_is_all_or_nothing():
    a = P.BlockAllocator(5, 4)
    s = a.create_sequence()
    a.append_tokens([s], [12])
    f = a.fork(s)
    g = a.fork(s)
    old = a.block_table(s)
    with pytest.raises(P.ExhaustedError):
        a.unshare([f, g])  # six blocks, two free
    with pytest.raises(P.PkvError):
        a.unshare([f, f])
    with pytest.raises(P.PkvError):
        a.unshare([f, 77])
    assert a.block_table(f) == old and a.block_table(g) == old and a.num_free == 2
    assert all(a.refcount(b) == 3 for b in old)


FAKE = 1 << 20  # never dereferenced: every call below is refused on the host


def _c16(hkv=2, d=64, bs=16, dtype=0):
    return _native.PkvCache(FAKE, FAKE, 8, bs, hkv, d, dtype)


def _c8(hkv=4, d=128, bs=16):
    return _native.PkvCacheI8(FAKE, FAKE, FAKE, FAKE, 8, bs, hkv, d, 0)


def _select(**k):
    a = dict(w=FAKE, ss=200, sh=100, keys=100, lens=FAKE, n=3, hkv=2, budget=8, sink=2, recent=2, kept=FAKE, new=FAKE + 64)
    a.update(k)
    return _native.lib().pkv_evict_select(a["w"], a["ss"], a["sh"], a["keys"], a["lens"], a["n"], a["hkv"], a["budget"],
                                          a["sink"], a["recent"], a["kept"], a["new"], None, None)


@pytest.mark.parametrize("change,status", [
    (dict(budget=0), 1), (dict(budget=-3), 1), (dict(sink=-1), 1), (dict(recent=-1), 1), (dict(sink=5, recent=4), 1),
    (dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), 1), (dict(n=-1), 1), (dict(hkv=0), 1), (dict(w=None), 1),
    (dict(lens=None), 1), (dict(kept=None), 1), (dict(new=None), 1), (dict(new=FAKE), 1), (dict(w=FAKE + 2), 1),
    (dict(keys=-1), 3), (dict(keys=1 << 31, sh=1 << 31, ss=1 << 33), 3), (dict(sh=99), 3), (dict(ss=199), 3),
    (dict(n=1 << 27), 9), (dict(n=0, w=None, lens=None, kept=None, new=None), 0)])
def test_select_refusals(change, status):
    assert _select(**change) == status, _native.lib().pkv_last_error()


def _compact(cache, i8=False, **k):
    a = dict(tables=FAKE, mb=4, lens=FAKE, n=3, kept=FAKE, budget=8, w=FAKE, ss=64 * cache.num_kv_heads, sh=64)
    a.update(k)
    f = _native.lib().pkv_evict_compact_int8 if i8 else _native.lib().pkv_evict_compact
    return f(ctypes.byref(cache), a["tables"], a["mb"], a["lens"], a["n"], a["kept"], a["budget"], a["w"], a["ss"], a["sh"],
             None, None)


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("change,status", [
    (dict(budget=0), 1), (dict(n=-1), 1), (dict(mb=-1), 1), (dict(tables=None), 1), (dict(lens=None), 1),
    (dict(kept=None), 1), (dict(w=FAKE + 1), 1), (dict(sh=63), 3), (dict(ss=64), 3), (dict(mb=1 << 27, w=None), 3),
    (dict(n=0, tables=None, lens=None, kept=None), 0)])
def test_compact_refusals(i8, change, status):
    assert _compact(_c8() if i8 else _c16(), i8, **change) == status, _native.lib().pkv_last_error()


def test_compact_refuses_shapes_it_was_not_built_for():
    assert _compact(_c16(d=96)) == 9
    assert _compact(_c16(bs=8), sh=64, ss=128) == 9
    assert _compact(_c16(bs=272)) == 9
    assert _compact(_c16(dtype=2)) == 2
    assert _compact(_c8(d=64), True) == 9
    assert _compact(_c8(bs=24), True) == 9
    f = _native.lib().pkv_evict_compact
    assert f(None, FAKE, 4, FAKE, 3, FAKE, 8, None, 0, 0, None, None) == 1


def _weights(i8=False, **k):
    hkv, d = (4, 128) if i8 else (2, 64)
    a = dict(hq=2 * hkv, w=FAKE, ss=64 * hkv, sh=64, out_dtype=2, ws=FAKE, ws_bytes=0, n=3, mb=4)
    a.update(k)
    c = _c8() if i8 else _c16()
    f = _native.lib().pkv_attn_decode_int8_weights if i8 else _native.lib().pkv_attn_decode_weights
    return f(FAKE, a["hq"] * d, ctypes.byref(c), FAKE, a["mb"], FAKE, a["n"], a["hq"], 1.0, 0, a["w"], a["ss"], a["sh"],
             FAKE, a["out_dtype"], a["ws"], a["ws_bytes"], None, None)


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("change,status", [
    (dict(w=None), 1), (dict(w=FAKE + 2), 1), (dict(sh=63), 3), (dict(ss=100), 3), (dict(hq=5), 3), (dict(out_dtype=1), 2),
    (dict(mb=1 << 27, sh=1 << 33, ss=1 << 36), 3), (dict(mb=1 << 26, sh=1 << 33, ss=1 << 36, n=1 << 12), 9),
    (dict(n=0, w=None), 0)])
def test_weights_refusals(i8, change, status):
    assert _weights(i8, **change) == status, _native.lib().pkv_last_error()


MANY = (1 << 30) + 16  # positions are 32-bit: a row of more than 2^30 keys, or a budget above that, is refused


def test_rows_past_2_30_keys_are_refused():
    assert _select(keys=MANY, sh=MANY, ss=2 * MANY) == 3
    assert _select(budget=MANY) == 3 and _select(budget=2 ** 31 - 1) == 3
    for i8 in (False, True):
        c = _c8() if i8 else _c16()
        assert _compact(c, i8, mb=MANY // 16, w=None) == 3
        assert _compact(c, i8, budget=MANY) == 3 and _compact(c, i8, budget=2 ** 31 - 1) == 3
        assert _weights(i8, mb=MANY // 16, sh=1 << 33, ss=1 << 36) == 3
    n = ctypes.c_size_t()
    assert _native.lib().pkv_attn_decode_weights_workspace_size(1, 8, 4, 128, MANY, 0, ctypes.byref(n)) != 0


def _varlen8(cache=None, **k):
    a = dict(q=FAKE, stride=8 * 128, tables=FAKE, mb=4, cu=FAKE, lens=FAKE, n=3, total=9, longest=4, hq=8, out=FAKE, dtype=2,
             ws=FAKE, ws_bytes=0)
    a.update(k)
    return _native.lib().pkv_attn_varlen_int8(a["q"], a["stride"], ctypes.byref(cache or _c8()), a["tables"], a["mb"], a["cu"],
                                              a["lens"], a["n"], a["total"], a["longest"], a["hq"], 1.0, 1, 0, a["out"],
                                              a["dtype"], a["ws"], a["ws_bytes"], None, None)


@pytest.mark.parametrize("change,status", [
    (dict(n=-1), 1), (dict(total=-1), 1), (dict(longest=-1), 1), (dict(mb=-1), 1), (dict(q=None), 1), (dict(tables=None), 1),
    (dict(cu=None), 1), (dict(lens=None), 1), (dict(out=None), 1), (dict(out=FAKE + 8), 1), (dict(q=FAKE + 4), 1),
    (dict(stride=8 * 128 - 2), 1), (dict(hq=6), 3), (dict(hq=12), 9), (dict(dtype=1), 2), (dict(n=65536), 9),
    (dict(n=0), 0), (dict(total=0, q=None, cu=None), 0)])
def test_varlen_int8_refusals(change, status):
    assert _varlen8(**change) == status, _native.lib().pkv_last_error()


def test_varlen_int8_refuses_caches_it_was_not_built_for():
    assert _varlen8(_c8(d=64), stride=8 * 64) == 9
    assert _varlen8(_c8(hkv=2)) == 9
    assert _varlen8(_c8(bs=24)) == 9
