"""A cache bounded by accumulated attention weight, on the GPU: the selection
and the moves bit for bit against a plain implementation, the key weights of a
decode call against binary64, and the operators together."""
import math

import numpy as np
import pytest
import torch

import oracle
import pagedattention_decode_gb300 as P
import workloads as W
from tests.cases import assert_close, decode_case

pytestmark = pytest.mark.gpu


def _err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---- selection -----------------------------------------------------------------

def _select(w, lens, budget, sink, recent):
    """Plain selection: kept [B, H, budget] and new lengths (numpy, stable sorts)."""
    B, H, _ = w.shape
    kept = np.full((B, H, budget), -1, np.int32)
    for s, L in enumerate(lens):
        n = min(L, budget)
        for h in range(H):
            if L <= budget:
                kept[s, h, :n] = np.arange(n)
                continue
            x = w[s, h, :L].astype(np.float64)
            rank = np.where(np.isnan(x), 2.0, np.where(np.isposinf(x), 1.0, 0.0))     # NaN over +inf over the rest
            x = np.where(np.isfinite(x) | np.isneginf(x), x, 0.0)
            ends = (np.arange(L) < sink) | (np.arange(L) >= L - recent)
            order = np.lexsort((np.arange(L), -x, -rank, ~ends))                       # the last key sorts first
            kept[s, h, :n] = np.sort(order[:n])
    return kept, np.minimum(np.array(lens), budget).astype(np.int32)


def _check_select(w, lens, budget, sink=0, recent=0, dev=None):
    dw = torch.from_numpy(w).cuda() if dev is None else dev
    err = _err()
    kept, new = P.evict_select(dw, torch.tensor(lens, dtype=torch.int32, device="cuda"), budget, sink=sink,
                               recent=recent, err=err)
    want, want_new = _select(w, lens, budget, sink, recent)
    assert int(err) == 0
    assert np.array_equal(new.cpu().numpy(), want_new)
    assert np.array_equal(kept.cpu().numpy(), want)


@pytest.mark.parametrize("budget,sink,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (7, 0, 0), (32, 4, 8), (64, 32, 32),
                                                (333, 1, 100), (1000, 4, 0)])
def test_select_lengths(budget, sink, recent):
    lens = [0, 1, 2, budget - 1, budget, budget + 1, 31, 32, 33, 1023, 1024, 1025, 2500]
    w = np.random.default_rng(budget).exponential(1.0, (len(lens), 3, 2560)).astype(np.float32)
    _check_select(w, [max(0, L) for L in lens], budget, sink, recent)


@pytest.mark.parametrize("kind", ["equal", "zeros", "few", "tail", "specials", "negative", "tiny"])
def test_select_values(kind):
    """Ties go to the lowest position; NaN, infinities, both zeros, denormals and negative weights order as documented."""
    r = np.random.default_rng(3)
    lens = [50, 700, 1500]
    w = np.zeros((3, 2, 1500), np.float32)
    if kind == "equal":
        w += 0.37
    elif kind == "few":
        w = r.integers(0, 3, w.shape).astype(np.float32)
    elif kind == "tail":
        w[:, :, 40:] = 1e-3
    elif kind == "specials":
        w = r.choice(np.array([np.nan, -np.nan, np.inf, -np.inf, 0.0, -0.0, 1.0, -1.0], np.float32), w.shape)
    elif kind == "negative":
        w = -r.exponential(1.0, w.shape).astype(np.float32)
    elif kind == "tiny":
        w = (r.integers(-5, 6, w.shape) * np.float32(1e-45)).astype(np.float32)
    for budget, sink, recent in [(20, 0, 0), (49, 3, 9), (600, 4, 64)]:
        _check_select(w, lens, budget, sink, recent)


@pytest.mark.parametrize("L", [9000, 40000, 131072, 300001])
def test_select_long(L):
    r = np.random.default_rng(L)
    w = np.exp(r.standard_normal((1, 2, L)) * 2).astype(np.float32)
    w[0, 1] = np.round(w[0, 1] * 4) / 4       # many ties
    _check_select(w, [L], 4097, 4, 512)
    _check_select(w, [L], L - 3, 0, 0)


def test_select_strides_and_reuse():
    """Weights as a view with its own strides; the same output buffers twice (a shorter row clears its tail)."""
    big = torch.rand(3, 5, 2 * 77 + 40, device="cuda")
    view = big[:, 1:4, 40:40 + 77]
    _check_select(view.cpu().numpy().copy(), [77, 3, 50], 16, 1, 2, dev=view)
    kept = torch.full((3, 3, 16), 99, dtype=torch.int32, device="cuda")
    new = torch.full((3,), 99, dtype=torch.int32, device="cuda")
    for lens in ([77, 70, 60], [0, 3, 17]):
        a, b = P.evict_select(view, torch.tensor(lens, dtype=torch.int32, device="cuda"), 16, kept=kept, new_lens=new)
        assert a is kept and b is new
        want, wn = _select(view.cpu().numpy(), lens, 16, 0, 0)
        assert np.array_equal(kept.cpu().numpy(), want) and np.array_equal(new.cpu().numpy(), wn)


def test_select_bad_lengths_are_flagged():
    w = torch.rand(3, 2, 64, device="cuda")
    err = _err()
    kept, new = P.evict_select(w, torch.tensor([65, 40, -1], dtype=torch.int32, device="cuda"), 8, err=err)
    assert int(err) == P.DEVERR["length"]
    assert (kept[0] == -1).all() and (kept[2] == -1).all() and new.tolist() == [65, 8, -1]
    assert np.array_equal(kept[1].cpu().numpy(), _select(w[1:2].cpu().numpy(), [40], 8, 0, 0)[0][0])


def test_select_no_sequences():
    kept, new = P.evict_select(torch.empty(0, 2, 64, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"), 8)
    assert kept.shape == (0, 2, 8) and new.shape == (0,)


# ---- moves ---------------------------------------------------------------------

def _random_kept(r, lens, hkv, budget):
    kept = np.full((len(lens), hkv, budget), -1, np.int32)
    for s, L in enumerate(lens):
        for h in range(hkv):
            n = min(L, budget)
            kept[s, h, :n] = np.sort(r.permutation(L)[:n])
    return kept


def _compact(pools, scales, w, tables, lens, kept, budget):
    """Plain moves (numpy, in place): pools uint16, or int8 with float32 scales."""
    bs = pools[0].shape[1]
    for s, L in enumerate(lens):
        if L <= budget:
            continue
        tab = tables[s]
        for h in range(kept.shape[1]):
            src = kept[s, h]
            dst = np.arange(budget)
            for which, x in enumerate(pools):
                rows = x[tab[src // bs], src % bs, h].copy()
                if scales is None:
                    x[tab[dst // bs], dst % bs, h] = rows
                    continue
                sc = scales[which]
                vals = rows.astype(np.float32) * sc[tab[src // bs], h][:, None]
                for b in range((budget + bs - 1) // bs):
                    sel = dst // bs == b
                    if np.array_equal(src[sel], dst[sel]):
                        continue
                    scale = np.float32(np.abs(vals[sel]).max()) * (np.float32(1) / np.float32(127))
                    q = np.clip(np.rint(vals[sel] / scale), -127, 127) if scale > 0 else np.zeros_like(vals[sel])
                    x[tab[b], dst[sel] % bs, h] = q.astype(np.int8)
                    sc[tab[b], h] = scale
            if w is not None:
                v = w[s, h, src].copy()
                w[s, h, :L] = 0
                w[s, h, :budget] = v


def _tables(r, lens, bs, spare=3):
    need = [-(-L // bs) for L in lens]
    nb = sum(need) + spare
    perm = r.permutation(nb)
    tab = np.full((len(lens), max(need + [1]) + 1), -1, np.int32)
    at = 0
    for i, n in enumerate(need):
        tab[i, :n] = perm[at:at + n]
        at += n
    return tab, nb


@pytest.mark.parametrize("hkv,d,bs,dtype", [(2, 64, 16, torch.float16), (8, 128, 16, torch.bfloat16), (3, 128, 48, torch.float16),
                                            (12, 64, 64, torch.bfloat16), (1, 128, 256, torch.float16)])
@pytest.mark.parametrize("budget", [1, 40, 300, 777])
def test_compact_bits(hkv, d, bs, dtype, budget):
    r = np.random.default_rng(budget + d + bs)
    lens = [0, 1, budget, budget + 1, 2 * budget + 5, 1500]
    tab, nb = _tables(r, lens, bs)
    pools = [r.integers(0, 1 << 16, (nb, bs, hkv, d)).astype(np.uint16) for _ in range(2)]
    kept = _random_kept(r, lens, hkv, budget)
    w = r.random((len(lens), hkv, tab.shape[1] * bs)).astype(np.float32)
    dev = [torch.from_numpy(x.view(np.int16).copy()).cuda().view(dtype) for x in pools]
    dw, err = torch.from_numpy(w.copy()).cuda(), _err()
    P.evict_compact(*dev, torch.from_numpy(tab).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                    torch.from_numpy(kept).cuda(), key_weights=dw, err=err)
    _compact(pools, None, w, tab, lens, kept, budget)
    assert int(err) == 0
    for a, b in zip(dev, pools):
        assert np.array_equal(a.view(torch.int16).cpu().numpy().view(np.uint16), b)
    assert np.array_equal(dw.cpu().numpy(), w)


@pytest.mark.parametrize("L,budget", [(5000, 2500), (40000, 1000), (40000, 30000)])
def test_compact_few_long_sequences(L, budget):
    """Few units of work, each split over several CTAs: dense keeps (every chunk overlaps its source) and sparse ones."""
    r = np.random.default_rng(L + budget)
    tab, nb = _tables(r, [L], 16)
    pools = [r.integers(0, 1 << 16, (nb, 16, 2, 64)).astype(np.uint16) for _ in range(2)]
    kept = _random_kept(r, [L], 2, budget)
    kept[0, 1] = np.arange(L - budget, L)                      # a shift by a constant
    w = r.random((1, 2, tab.shape[1] * 16)).astype(np.float32)
    dev = [torch.from_numpy(x.view(np.int16).copy()).cuda().view(torch.float16) for x in pools]
    dw = torch.from_numpy(w.copy()).cuda()
    P.evict_compact(*dev, torch.from_numpy(tab).cuda(), torch.tensor([L], dtype=torch.int32, device="cuda"),
                    torch.from_numpy(kept).cuda(), key_weights=dw)
    _compact(pools, None, w, tab, [L], kept, budget)
    for a, b in zip(dev, pools):
        assert np.array_equal(a.view(torch.int16).cpu().numpy().view(np.uint16), b)
    assert np.array_equal(dw.cpu().numpy(), w)


@pytest.mark.parametrize("hkv,bs", [(4, 16), (8, 32), (4, 48), (1, 240), (4, 256)])
@pytest.mark.parametrize("budget", [1, 40, 300, 777])
def test_compact_int8_bits(hkv, bs, budget):
    r = np.random.default_rng(budget + bs)
    lens = [0, 1, budget, budget + 1, 2 * budget + 5, 1500]
    tab, nb = _tables(r, lens, bs)
    pools = [r.integers(-127, 128, (nb, bs, hkv, 128)).astype(np.int8) for _ in range(2)]
    scales = [np.exp(r.standard_normal((nb, hkv))).astype(np.float32) * np.float32(0.02) for _ in range(2)]
    for sc in scales:
        sc[r.random(sc.shape) < 0.1] = 0                        # all-zero blocks
    kept = _random_kept(r, lens, hkv, budget)
    kept[5, 0, :budget] = np.arange(budget)                     # a head in which nothing moves
    w = r.random((len(lens), hkv, tab.shape[1] * bs)).astype(np.float32)
    dev = [torch.from_numpy(x.copy()).cuda() for x in pools + scales]
    dw, err = torch.from_numpy(w.copy()).cuda(), _err()
    P.evict_compact_int8(*dev, torch.from_numpy(tab).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                         torch.from_numpy(kept).cuda(), key_weights=dw, err=err)
    _compact(pools, scales, w, tab, lens, kept, budget)
    assert int(err) == 0
    for a, b in zip(dev, pools + scales):
        assert np.array_equal(a.cpu().numpy(), b)
    assert np.array_equal(dw.cpu().numpy(), w)


@pytest.mark.parametrize("L,budget", [(6000, 3000), (20000, 16000)])
def test_compact_int8_few_long_sequences(L, budget):
    r = np.random.default_rng(L)
    tab, nb = _tables(r, [L], 32)
    pools = [r.integers(-127, 128, (nb, 32, 4, 128)).astype(np.int8) for _ in range(2)]
    scales = [np.exp(r.standard_normal((nb, 4))).astype(np.float32) for _ in range(2)]
    kept = _random_kept(r, [L], 4, budget)
    dev = [torch.from_numpy(x.copy()).cuda() for x in pools + scales]
    P.evict_compact_int8(*dev, torch.from_numpy(tab).cuda(), torch.tensor([L], dtype=torch.int32, device="cuda"),
                         torch.from_numpy(kept).cuda())
    _compact(pools, scales, None, tab, [L], kept, budget)
    for a, b in zip(dev, pools + scales):
        assert np.array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("i8", [False, True])
def test_compact_bad_data_is_flagged_and_stays_in_bounds(i8):
    """Kept positions that fall, repeat, run backwards or leave the sequence, and a block id outside the pool: the error
    word says so, other sequences move as they should."""
    r = np.random.default_rng(8)
    hkv, d, bs, budget, L = 4, 128, 16, 20, 50
    lens = [L] * 7
    tab, nb = _tables(r, lens, bs)
    kept = _random_kept(r, lens, hkv, budget)
    tables = tab.copy()
    kept[0, 0, 5] = kept[0, 0, 4]       # repeats
    kept[1, 1, 6] = L                   # past the end
    kept[2, 2, 7] = 3                   # backwards
    kept[3, 3, 8] = -1
    tables[4, 0] = nb                   # bad block
    lens[5] = tab.shape[1] * bs + 1     # longer than its table
    if i8:
        pools = [r.integers(-127, 128, (nb, bs, hkv, d)).astype(np.int8) for _ in range(2)]
        scales = [r.random((nb, hkv)).astype(np.float32) + np.float32(0.1) for _ in range(2)]
        dev = [torch.from_numpy(x.copy()).cuda() for x in pools + scales]
        call = P.evict_compact_int8
    else:
        pools = [r.integers(0, 1 << 16, (nb, bs, hkv, d)).astype(np.uint16) for _ in range(2)]
        scales = None
        dev = [torch.from_numpy(x.view(np.int16).copy()).cuda().view(torch.float16) for x in pools]
        call = P.evict_compact
    err = _err()
    call(*dev, torch.from_numpy(tables).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
         torch.from_numpy(kept).cuda(), err=err)
    assert int(err) == P.DEVERR["keep"] | P.DEVERR["block"] | P.DEVERR["length"]
    before = [x.copy() for x in pools + (scales or [])]
    _compact(pools, scales, None, tab[6:], lens[6:], kept[6:], budget)
    for a, b, old in zip(dev, pools + (scales or []), before):
        got = a.view(torch.int16).cpu().numpy().view(np.uint16) if a.dtype == torch.float16 else a.cpu().numpy()
        ids = tab[6][:4]
        assert np.array_equal(got[ids], b[ids])
        ids = tab[5][:4]
        assert np.array_equal(got[ids], old[ids])


# ---- key weights -----------------------------------------------------------------

def _weights64(q, k, scale, dtype_rows):
    """Softmax weights of one sequence and KV head, q [G, D], k [L, D] binary64 -> [L] summed over the rows, and the
    bound on a computed weight's relative error: a score is a sum of D products (error <= D 2^-23 sum |q k| scale for
    sums that truncate), scaled twice (2 2^-24 |score|, taken with the sum), the maximum's error and the sum's (L adds at
    worst) come on top, exp2 and the division 2^-21 together."""
    s = scale * q @ k.T
    mag = scale * np.abs(q) @ np.abs(k).T
    e = np.exp(s - s.max(1, keepdims=True))
    p = e / e.sum(1, keepdims=True)
    d = (q.shape[1] + 2) * 2.0 ** -23 * mag.max()
    return p.sum(0), math.expm1(2 * d) + k.shape[0] * 2.0 ** -24 + 2.0 ** -21


def _rows(pool, table, L, h):
    bs = pool.shape[1]
    t = np.arange(L)
    return pool[table[t // bs], t % bs, h]


@pytest.mark.parametrize("hq,hkv,d,bs,dtype", [(12, 12, 64, 16, "f16"), (32, 8, 128, 16, "bf16"), (8, 4, 64, 32, "bf16"),
                                               (16, 2, 128, 48, "f16"), (4, 4, 128, 16, "f16"), (6, 3, 128, 64, "f16"),
                                               (64, 8, 64, 16, "f16")])
@pytest.mark.parametrize("window", [0, 1, 100])
def test_key_weights_match_binary64(hq, hkv, d, bs, dtype, window):
    lens = [0, 1, 15, 16, 17, 300, 1111, 5000]
    c = decode_case(70 + hq + d, lens, hq, hkv, d, bs, dtype)
    dev = c.to("cuda")
    keys = c.tables.shape[1] * bs
    w0 = torch.rand(len(lens), hkv, keys + 5, generator=torch.Generator().manual_seed(1))
    dw, err = w0.cuda(), _err()
    out = P.attn_decode(dev.q, dev.k_cache, dev.v_cache, dev.tables, dev.lens, c.scale, window=window, key_weights=dw, err=err)
    plain = P.attn_decode(dev.q, dev.k_cache, dev.v_cache, dev.tables, dev.lens, c.scale, window=window)
    assert int(err) == 0 and torch.equal(out, plain)
    got = dw.cpu().double().numpy()
    k = c.k_cache.double().numpy()
    g = hq // hkv
    for s, L in enumerate(lens):
        lo = max(0, L - window) if window else 0
        assert np.array_equal(got[s, :, L:], w0[s, :, L:].double().numpy())
        assert np.array_equal(got[s, :, :lo], w0[s, :, :lo].double().numpy())
        for h in range(hkv):
            if L == 0:
                continue
            p, rel = _weights64(c.q[s, h * g:(h + 1) * g].double().numpy(), _rows(k, c.tables[s].numpy(), L, h)[lo:], c.scale, None)
            want = w0[s, h, lo:L].double().numpy() + p
            assert (np.abs(got[s, h, lo:L] - want) <= rel * p + 2.0 ** -24 * want).all()


def test_key_weights_sum_to_the_heads_and_do_not_depend_on_the_run():
    """Each call adds G per (sequence, KV head) in all; two calls on two copies give the same bits (no atomics)."""
    c = decode_case(5, [4000, 130, 7], 32, 8, 128, 16, "bf16").to("cuda")
    keys = c.tables.shape[1] * 16
    a, b = torch.zeros(3, 8, keys, device="cuda"), torch.zeros(3, 8, keys, device="cuda")
    for w in (a, b):
        for _ in range(3):
            P.attn_decode(c.q, c.k_cache, c.v_cache, c.tables, c.lens, c.scale, key_weights=w)
    assert torch.equal(a, b)
    # 3 calls x 4 heads; binary32 sums of up to 4,000 weights, each off by at most ~1e-5 of itself
    assert torch.allclose(a.double().sum(-1), torch.full((3, 8), 12.0, device="cuda", dtype=torch.float64), rtol=1e-4)


@pytest.mark.parametrize("hq,hkv,bs,dtype", [(32, 8, 16, "f16"), (8, 4, 32, "bf16"), (4, 4, 48, "f16"), (32, 4, 16, "bf16")])
@pytest.mark.parametrize("window", [0, 64])
def test_key_weights_int8(hq, hkv, bs, dtype, window):
    r = np.random.default_rng(hq + bs)
    lens = [0, 1, 17, 500, 3001]
    tab, nb = _tables(r, lens, bs)
    kq, vq = (r.integers(-127, 128, (nb, bs, hkv, 128)).astype(np.int8) for _ in range(2))
    ks, vs = ((r.random((nb, hkv)) * 0.02 + 0.015).astype(np.float32) for _ in range(2))
    q = torch.from_numpy(r.standard_normal((len(lens), hq, 128))).to(W.DTYPES[dtype])
    keys = tab.shape[1] * bs
    dw, err = torch.zeros(len(lens), hkv, keys, device="cuda"), _err()
    scale = 128 ** -0.5
    args = [torch.from_numpy(x).cuda() for x in (kq, vq, ks, vs, tab)]
    out = P.attn_decode_int8(q.cuda(), *args, torch.tensor(lens, dtype=torch.int32, device="cuda"), scale, window=window,
                             key_weights=dw, err=err)
    want = oracle.paged_attention_int8(q, dtype, kq, vq, ks, vs, tab, np.array(lens, np.int32), scale, window=window)
    assert int(err) == 0
    assert_close(out, want)
    got = dw.cpu().double().numpy()
    k = kq.astype(np.float64) * ks.astype(np.float64)[:, None, :, None]
    g = hq // hkv
    for s, L in enumerate(lens):
        lo = max(0, L - window) if window else 0
        assert not got[s, :, L:].any() and not got[s, :, :lo].any()
        for h in range(hkv):
            if L:
                p, rel = _weights64(q[s, h * g:(h + 1) * g].double().numpy(), _rows(k, tab[s], L, h)[lo:], scale, None)
                assert (np.abs(got[s, h, lo:L] - p) <= rel * p + 2.0 ** -24 * p).all()


def test_key_weights_strided_rows_and_side_stream():
    """Weights as rows of a larger tensor, query rows with a stride, the call on a stream of its own."""
    c = decode_case(9, [100, 40], 8, 4, 64, 16).to("cuda")
    keys = c.tables.shape[1] * 16
    big = torch.zeros(2, 6, keys + 30, device="cuda")
    view = big[:, 1:5, 3:3 + keys]
    wide = torch.zeros(2, 10, 64, dtype=torch.float16, device="cuda")
    wide[:, :8] = c.q
    plain = torch.zeros(2, 4, keys, device="cuda")
    P.attn_decode(c.q, c.k_cache, c.v_cache, c.tables, c.lens, c.scale, key_weights=plain)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(P.decode_workspace_size(2, 8, 4, 64, max_keys=keys), dtype=torch.uint8, device="cuda")
    P.attn_decode(wide[:, :8], c.k_cache, c.v_cache, c.tables, c.lens, c.scale, key_weights=view, workspace=ws, stream=st)
    st.synchronize()
    assert torch.equal(view, plain)
    view.zero_()
    assert not big.any()


def test_refusals():
    c = decode_case(9, [100, 40], 8, 4, 64, 16).to("cuda")
    keys = c.tables.shape[1] * 16
    w = torch.zeros(2, 4, keys, device="cuda")

    def call(**k):
        a = dict(key_weights=w)
        a.update(k)
        P.attn_decode(c.q, c.k_cache, c.v_cache, c.tables, c.lens, c.scale, **a)

    call()
    for bad, kind in [(dict(key_weights=w.half()), TypeError), (dict(key_weights=w[0]), TypeError),
                      (dict(key_weights=w.cpu()), TypeError), (dict(key_weights=w[:, :, :-1]), ValueError),
                      (dict(key_weights=w[:1]), ValueError), (dict(key_weights=w[:, :3]), ValueError),
                      (dict(key_weights=torch.zeros(2, 4, 2 * keys, device="cuda")[:, :, ::2]), ValueError),
                      (dict(key_weights=torch.zeros(4, 2, keys, device="cuda").transpose(0, 1)), P.PkvError),
                      (dict(k_new=c.q[:, :4], v_new=c.q[:, :4]), ValueError),
                      (dict(workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda")[:256]), P.PkvError),
                      (dict(out=torch.empty(2, 8, 64, device="cuda", dtype=torch.float64)), ValueError),
                      (dict(err=torch.zeros(1, device="cuda")), TypeError)]:
        with pytest.raises(kind):
            call(**bad)
    lens = c.lens
    for bad, kind in [(dict(budget=0), ValueError), (dict(sink=5, recent=4), ValueError), (dict(sink=-1), ValueError),
                      (dict(seq_lens=lens[:1]), ValueError), (dict(seq_lens=lens.long()), TypeError),
                      (dict(key_weights=w.double()), TypeError), (dict(new_lens=lens), P.PkvError),
                      (dict(kept=torch.zeros(2, 4, 9, dtype=torch.int32, device="cuda")), ValueError)]:
        a = dict(key_weights=w, seq_lens=lens, budget=8)
        a.update(bad)
        with pytest.raises(kind):
            P.evict_select(**a)
    kept = torch.zeros(2, 4, 8, dtype=torch.int32, device="cuda")
    for bad, kind in [(dict(kept=kept[:1]), ValueError), (dict(kept=kept[:, :2].contiguous()), ValueError), (dict(kept=kept.long()), TypeError),
                      (dict(seq_lens=lens[:1]), ValueError), (dict(block_tables=c.tables[:1]), ValueError),
                      (dict(key_weights=w[:, :, :20]), ValueError), (dict(k_cache=c.k_cache[:2]), ValueError)]:
        a = dict(k_cache=c.k_cache, v_cache=c.v_cache, block_tables=c.tables, seq_lens=lens, kept=kept)
        a.update(bad)
        with pytest.raises(kind):
            P.evict_compact(**a)


def test_offsets_past_32_bits():
    """Pools of more than 2^32 bytes and weights whose rows lie 2^31 entries apart: decode with weights, selection, moves."""
    hq, hkv, d, bs = 8, 8, 128, 16
    nb = (1 << 32) // (bs * hkv * d * 2) + 64                   # 4.3 GB each
    gen = torch.Generator(device="cuda").manual_seed(3)
    kc, vc = (torch.empty(nb, bs, hkv, d, dtype=torch.float16, device="cuda") for _ in range(2))
    L, budget = 150, 40
    ids = torch.tensor([[nb - 1 - 3 * i for i in range(10)], [nb - 2 - 3 * i for i in range(10)]], dtype=torch.int32, device="cuda")
    for x in (kc, vc):
        x[ids.long()] = torch.randn(2, 10, bs, hkv, d, generator=gen, device="cuda").half()
    far = torch.zeros((1 << 31) + hkv * 160, device="cuda")
    w = far.as_strided((2, hkv, 160), (1 << 31, 160, 1))
    near = torch.zeros(2, hkv, 160, device="cuda")
    lens = torch.tensor([L, L - 7], dtype=torch.int32, device="cuda")
    q = torch.randn(2, hq, d, generator=gen, device="cuda").half()
    # the same sequences in a small pool
    small = torch.arange(20, dtype=torch.int32, device="cuda").view(2, 10)
    ks, vs = kc[ids.long()].reshape(20, bs, hkv, d).clone(), vc[ids.long()].reshape(20, bs, hkv, d).clone()
    a = P.attn_decode(q, kc, vc, ids, lens, d ** -0.5, key_weights=w)
    b = P.attn_decode(q, ks, vs, small, lens, d ** -0.5, key_weights=near)
    assert torch.equal(a, b) and torch.equal(w, near)
    kept, _ = P.evict_select(w, lens, budget)
    assert torch.equal(kept, P.evict_select(near, lens, budget)[0])
    P.evict_compact(kc, vc, ids, lens, kept, key_weights=w)
    P.evict_compact(ks, vs, small, lens, kept, key_weights=near)
    assert torch.equal(w, near)
    assert torch.equal(kc[ids.long()].reshape(20, bs, hkv, d), ks) and torch.equal(vc[ids.long()].reshape(20, bs, hkv, d), vs)


def test_two_calls_at_once():
    """Decode with weights, selection and moves of two batches on two streams, each with its own workspace."""
    cases = [decode_case(60 + i, [900, 300, 31], 16, 8, 128, 16, "f16", poison=False).to("cuda") for i in range(2)]
    keys = [c.tables.shape[1] * 16 for c in cases]

    def run(c, n):
        w = torch.zeros(3, 8, n, device="cuda")
        ws = torch.empty(P.decode_workspace_size(3, 16, 8, 128, max_keys=n), dtype=torch.uint8, device="cuda")
        k, v = c.k_cache.clone(), c.v_cache.clone()
        for _ in range(5):
            out = P.attn_decode(c.q, k, v, c.tables, c.lens, c.scale, key_weights=w, workspace=ws)
        kept, new = P.evict_select(w, c.lens, 64, sink=2, recent=16)
        P.evict_compact(k, v, c.tables, c.lens, kept, key_weights=w)
        return out, w, kept, new, k, v

    alone = [run(c, n) for c, n in zip(cases, keys)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    both = []
    for c, n, st in zip(cases, keys, streams):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            both.append(run(c, n))
    torch.cuda.synchronize()
    for x, y in zip(alone, both):
        for a, b in zip(x, y):
            assert torch.equal(a, b)


# ---- together --------------------------------------------------------------------

def test_a_bounded_cache_over_many_steps():
    """Write, decode with weights, evict, go on: two layers, forked sequences made private, blocks given back.  After
    each cut, attention over the cache equals attention over the kept keys of the uncut one."""
    hq, hkv, d, bs, budget = 8, 4, 64, 16, 40
    layers, steps = 2, 70
    g = W.generator(77)
    a = P.BlockAllocator(64, bs)
    base = a.create_sequence()
    prompt = W.normal(g, (layers, 2, 60, hkv, d), 1.0, "f16")
    slots, _ = a.append_tokens([base], [60])
    kc = [torch.zeros(64, bs, hkv, d, dtype=torch.float16, device="cuda") for _ in range(layers)]
    vc = [torch.zeros_like(x) for x in kc]
    sl = torch.tensor(slots, dtype=torch.int64, device="cuda")
    for l in range(layers):
        P.write_kv(prompt[l, 0].cuda(), prompt[l, 1].cuda(), sl, kc[l], vc[l])
    seqs = [base, a.fork(base), a.fork(base)]
    pairs = a.unshare(seqs)
    assert len(pairs) == 2 * 4
    P.check_copy_pairs(pairs, 64)
    P.copy_blocks(kc, vc, torch.tensor(pairs, dtype=torch.int64, device="cuda"))
    mb = 8
    tables, lens = torch.empty(3, mb, dtype=torch.int32), torch.empty(3, dtype=torch.int32)
    w = [torch.zeros(3, hkv, mb * bs, device="cuda") for _ in range(layers)]
    # what each head still holds, per layer and sequence: rows of K and V in order
    held = [[[(prompt[l, 0][:, h].double(), prompt[l, 1][:, h].double()) for h in range(hkv)] for _ in seqs] for l in range(layers)]
    err = _err()
    cuts = 0
    for step in range(steps):
        slots, cow = a.append_tokens(seqs)
        assert cow == []
        sl = torch.tensor(slots, dtype=torch.int64, device="cuda")
        a.fill_tables(seqs, mb, tables, lens)
        dt, dl = tables.cuda(), lens.cuda()
        outs = []
        for l in range(layers):
            k, v, q = (W.normal(g, (3, n, d), 1.0, "f16") for n in (hkv, hkv, hq))
            P.write_kv(k.cuda(), v.cuda(), sl, kc[l], vc[l])
            out = P.attn_decode(q.cuda(), kc[l], vc[l], dt, dl, d ** -0.5, key_weights=w[l], err=err)
            for s in range(3):
                for h in range(hkv):
                    hk, hv = held[l][s][h]
                    hk, hv = torch.cat([hk, k[s, h][None].double()]), torch.cat([hv, v[s, h][None].double()])
                    held[l][s][h] = (hk, hv)
                    p = torch.softmax(q[s, 2 * h:2 * h + 2].double() @ hk.T * d ** -0.5, -1)
                    assert_close(out[s, 2 * h:2 * h + 2], (p @ hv).numpy(), what=f"step {step}")
        if int(lens[0]) >= budget + 24:
            cuts += 1
            for l in range(layers):
                kept, new = P.evict_select(w[l], dl, budget, sink=2, recent=8, err=err)
                P.evict_compact(kc[l], vc[l], dt, dl, kept, key_weights=w[l], err=err)
                idx = kept.long().cpu()
                for s in range(3):
                    for h in range(hkv):
                        hk, hv = held[l][s][h]
                        held[l][s][h] = (hk[idx[s, h]], hv[idx[s, h]])
            assert new.tolist() == [budget] * 3
            for s in seqs:
                a.truncate(s, budget)
    assert int(err) == 0 and cuts == 3
    assert all(len(a.block_table(s)) <= 4 for s in seqs)


def test_captured_and_replayed():
    """Decode with weights, selection and moves as one graph, replayed: the same bits as the calls."""
    c = decode_case(31, [200, 90, 64], 16, 8, 128, 16, "bf16", poison=False).to("cuda")
    keys = c.tables.shape[1] * 16
    ws = torch.empty(P.decode_workspace_size(3, 16, 8, 128, max_keys=keys), dtype=torch.uint8, device="cuda")
    start = [c.k_cache.clone(), c.v_cache.clone(), torch.rand(3, 8, keys, device="cuda")]
    bufs = [x.clone() for x in start]
    out = torch.empty(3, 16, 128, device="cuda")
    kept = torch.empty(3, 8, 48, dtype=torch.int32, device="cuda")
    new = torch.empty(3, dtype=torch.int32, device="cuda")

    def step():
        P.attn_decode(c.q, bufs[0], bufs[1], c.tables, c.lens, c.scale, out=out, key_weights=bufs[2], workspace=ws)
        P.evict_select(bufs[2], c.lens, 48, sink=1, recent=9, kept=kept, new_lens=new)
        P.evict_compact(bufs[0], bufs[1], c.tables, c.lens, kept, key_weights=bufs[2])

    graph = P.StepGraph(step)
    results = []
    for run in (step, graph.replay):
        for b, s in zip(bufs, start):
            b.copy_(s)
        for _ in range(3):
            run()
        torch.cuda.synchronize()
        results.append([x.clone() for x in (*bufs, out, kept, new)])
    for x, y in zip(*results):
        assert torch.equal(x.view(torch.int16) if x.dtype == torch.bfloat16 else x,
                           y.view(torch.int16) if y.dtype == torch.bfloat16 else y)


def test_what_a_call_on_another_stream_allocates_is_not_reused_under_it():
    """No workspace and no output given, a stream other than the current one with work queued on it: the current
    stream takes and clears memory meanwhile."""
    c = decode_case(41, [700, 90, 64, 1500], 16, 8, 128, 16, "f16", poison=False).to("cuda")
    w = torch.zeros(4, 8, c.tables.shape[1] * 16, device="cuda")
    want_w = w.clone()
    args = (c.q, c.k_cache, c.v_cache, c.tables, c.lens, c.scale)
    want = P.attn_decode(*args, key_weights=want_w)
    want_kept, want_lens = P.evict_select(want_w, c.lens, 80, sink=4, recent=16)
    size = P.decode_workspace_size(4, 16, 8, 128, max_keys=w.shape[2])
    a, b = (torch.randn(4096, 4096, device="cuda") for _ in range(2))
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(40):                      # some tens of milliseconds
            torch.mm(a, b, out=a)
            a.clamp_(-1, 1)
    out = P.attn_decode(*args, key_weights=w, stream=side)
    kept, lens = P.evict_select(w, c.lens, 80, sink=4, recent=16, stream=side)
    cleared = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert len(cleared) == 4
    assert torch.equal(out, want) and torch.equal(w, want_w)
    assert torch.equal(kept, want_kept) and torch.equal(lens, want_lens)
