"""Packed attention over an int8 cache (chunks on the tensor cores, decode rows
on the split-K kernel) against binary64, and the int8 cache's operators together."""
import math

import numpy as np
import pytest
import torch

import pagedattention_decode_gb300 as P
import workloads as W
from tests.cases import TOL

pytestmark = pytest.mark.gpu


def _case(seed, q_lens, kv_lens, hq, hkv, bs, dtype, k_size=0.02, v_size=0.02):
    r = np.random.default_rng(seed)
    need = [-(-L // bs) for L in kv_lens]
    nb = sum(need) + 3
    perm = r.permutation(nb)
    tab = np.full((len(kv_lens), max(need + [1]) + 1), -1, np.int32)
    at = 0
    for i, n in enumerate(need):
        tab[i, :n] = perm[at:at + n]
        at += n
    kq, vq = (r.integers(-128, 128, (nb, bs, hkv, 128)).astype(np.int8) for _ in range(2))
    ks = ((r.random((nb, hkv)) + 0.5) * k_size).astype(np.float32)
    vs = ((r.random((nb, hkv)) + 0.5) * v_size).astype(np.float32)
    unused = perm[at:]
    ks[unused] = np.nan                       # blocks that no sequence holds
    vs[unused] = np.nan
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    q = torch.from_numpy(r.standard_normal((int(cu[-1]), hq, 128))).to(W.DTYPES[dtype])
    return q, kq, vq, ks, vs, tab, cu, np.array(kv_lens, np.int32)


def _reference(q, kq, vq, ks, vs, tab, cu, lens, scale, causal=True, window=0, skip=()):
    """Binary64 outputs and the bound on a row's error: a weight's relative error (scores: sums of 128 products that
    truncate and two scalings, as in the key-weight tests; exp2 and the row sum) plus half a step of fp16, 2^-11, for a
    chunk's weights and 2^-24 per key of the accumulation, times sum p |v|; decode rows are held to the decode call's
    tolerance.  Below fp16's normal range a weight is off by 2^-25 at most: weights are p times the V scale in units of
    the largest of them, so a key's error is at most 2^-25 of the largest V scale times a code of at most 128; the
    folded log2 of a scale (off by 2^-24 of at most 128) is 2^-17 of each weight.  A row whose weights are all under
    2^-126 apart from the largest loses them: L 2^-126 times 128 codes."""
    bs, hkv = kq.shape[1], kq.shape[2]
    hq = q.shape[1]
    g = hq // hkv
    want = np.zeros(q.shape)
    bound = np.zeros(q.shape)
    qd = q.double().numpy()
    for s, L in enumerate(lens):
        a, b = int(cu[s]), int(cu[s + 1])
        n = b - a
        if n == 0 or L == 0 or s in skip:
            continue
        t = np.arange(L)
        blk = tab[s][t // bs]
        k = kq[blk, t % bs].astype(np.float64) * ks[blk].astype(np.float64)[:, :, None]
        v = vq[blk, t % bs].astype(np.float64) * vs[blk].astype(np.float64)[:, :, None]
        last = L - n + np.arange(n) if causal else np.full(n, L - 1)
        seen = t[None, :] <= last[:, None]
        if window:
            seen &= t[None, :] > last[:, None] - window
        for h in range(hq):
            x = scale * qd[a:b, h] @ k[:, h // g].T
            x = np.where(seen, x, -np.inf)
            e = np.exp(x - x.max(1, keepdims=True))
            p = e / e.sum(1, keepdims=True)
            want[a:b, h] = p @ v[:, h // g]
            mag = abs(scale) * (np.abs(qd[a:b, h]) @ np.abs(k[:, h // g]).T)[seen].max()
            rel = math.expm1(2 * 130 * 2.0 ** -23 * mag) + (2.0 ** -11 + 2.0 ** -17 if n > 1 else 2.0 ** -16) + (L + 4) * 2.0 ** -24
            tiny = L * 128 * (2.0 ** -126 + 2.0 ** -25 * float(vs[blk, h // g].max()))
            bound[a:b, h] = rel * (p @ np.abs(v[:, h // g])) + tiny + (TOL if n == 1 else 0)
    return want, bound


def _run(case, scale, err=None, **k):
    q, kq, vq, ks, vs, tab, cu, lens = case
    dev = [torch.from_numpy(x).cuda() for x in (kq, vq, ks, vs, tab, cu, lens)]
    n = int(np.diff(cu).max()) if len(cu) > 1 else 0
    return P.attn_varlen_int8(q.cuda(), *dev, n, scale, err=err, **k)


def _check(case, scale, got=None, **k):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = _run(case, scale, err=err, **k) if got is None else got
    opts = {a: b for a, b in k.items() if a in ("causal", "window")}
    want, bound = _reference(*case, scale, **opts)
    assert int(err) == 0
    o = out.cpu().double().numpy()
    if out.dtype != torch.float32:  # rounded once: half a step of the type
        bound = bound * (1 + 2.0 ** -8) + np.abs(want) * torch.finfo(out.dtype).eps / 2 + 2.0 ** -25
    assert np.isfinite(o).all()
    off = np.abs(o - want) - bound
    assert off.max() <= 0, (np.abs(o - want).max(), np.unravel_index(off.argmax(), off.shape))


MIX_Q = [1, 2, 0, 127, 128, 129, 1, 300, 5, 513, 64]
MIX_KV = [1, 2, 0, 127, 200, 129, 1000, 333, 2001, 1025, 64]


@pytest.mark.parametrize("hq,hkv,bs,dtype", [(32, 8, 16, "f16"), (32, 8, 32, "bf16"), (8, 8, 48, "f16"), (16, 8, 64, "bf16"),
                                             (32, 4, 256, "f16"), (24, 12, 16, "bf16"), (4, 4, 240, "bf16")])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 100), (True, 1), (False, 0), (False, 300)])
def test_against_binary64(hq, hkv, bs, dtype, causal, window):
    _check(_case(hq + bs, MIX_Q, MIX_KV, hq, hkv, bs, dtype), 128 ** -0.5, causal=causal, window=window)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_16_bit_outputs_and_strided_rows(dtype):
    case = _case(3, [70, 1, 200], [500, 90, 200], 16, 4, 16, dtype)
    _check(case, 128 ** -0.5, out_dtype=W.DTYPES[dtype])
    wide = torch.zeros(271, 20, 128, dtype=W.DTYPES[dtype])
    wide[:, :16] = case[0]
    dev = [torch.from_numpy(x).cuda() for x in case[1:]]
    ws = torch.empty(P.varlen_workspace_size(3, 16, 4, 128), dtype=torch.uint8, device="cuda")
    out = torch.full((271, 16, 128), float("nan"), device="cuda")
    got = P.attn_varlen_int8(wide.cuda()[:, :16], *dev, 200, 128 ** -0.5, out=out, workspace=ws)
    assert got is out
    _check(case, 128 ** -0.5, got=out)


@pytest.mark.parametrize("k_size,v_size,scale", [(2.0, 0.02, 128 ** -0.5), (0.02, 3e4, 128 ** -0.5), (0.02, 1e-7, 128 ** -0.5),
                                                 (0.02, 0.02, 0.0), (0.02, 0.02, -0.1), (1e-4, 0.02, 1.0)])
def test_ranges(k_size, v_size, scale):
    """Scores that move the running maximum by hundreds, V scales far outside 16-bit floats' comfortable range, a scale
    of zero and a negative one."""
    case = _case(17, [200, 3, 140], [900, 700, 140], 16, 4, 16, "f16", k_size, v_size)
    case[3][case[5][0, 40:50]] *= 30            # a late jump of the scores
    if k_size > 1:                              # scores of some hundred: exact enough only without the decode rows' tolerance
        case[3][case[5][0, 40:50]] /= 30
    _check(case, scale)


def test_zero_blocks_and_values_that_are_not_seen():
    """All-zero blocks (scale 0), and NaN scales in blocks that lie wholly before every row's window or past the keys."""
    case = _case(19, [40, 1], [1000, 500], 16, 4, 16, "bf16")
    q, kq, vq, ks, vs, tab, cu, lens = case
    for b in (0, 3, 60):
        blk = tab[0, b]
        kq[blk], vq[blk], ks[blk], vs[blk] = 0, 0, 0, 0
    _check(case, 128 ** -0.5)
    # row 0 of the chunk sees keys 861 .. 960: block 53 (848 .. 863) is the first one read
    ks[tab[0, :53]], vs[tab[0, :53]] = np.nan, np.nan
    ks[tab[1, :25]], vs[tab[1, :25]] = np.nan, np.nan
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = _run(case, 128 ** -0.5, err=err, window=100)
    clean = (q, kq, vq, np.nan_to_num(ks), np.nan_to_num(vs), tab, cu, lens)
    want, bound = _reference(*clean, 128 ** -0.5, window=100)
    assert int(err) == 0 and (np.abs(out.cpu().double().numpy() - want) <= bound).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("which", ["k", "v", "both"])
def test_scales_that_are_not_finite_stay_with_the_rows_that_see_them(which, bad):
    """A block of the chunk itself with such a scale: the rows before it are as if it were not there."""
    case = _case(29, [300], [420], 16, 4, 16, "f16")
    q, kq, vq, ks, vs, tab, cu, lens = case
    want, bound = _reference(*case, 128 ** -0.5)
    first = 20 * 16 - 120                      # the first row that sees a key of block 20
    blk = tab[0, 20]
    if which != "v":
        ks[blk] = bad
    if which != "k":
        vs[blk] = bad
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = _run(case, 128 ** -0.5, err=err).cpu().double().numpy()
    assert int(err) == 0 and (np.abs(out - want) <= bound)[:first].all()
    if which != "k" or math.isnan(bad):        # (an infinite K scale: scores of -inf leave a row finite)
        assert not np.isfinite(out[first:]).all(axis=-1).any()


def test_scales_of_any_sign_and_zero_over_codes():
    """Scales are plain factors: negative ones, zeros over codes that are not zero, and V scales from 1e-3 to 10 in one row."""
    case = _case(41, [150, 3], [600, 333], 16, 4, 16, "f16")
    r = np.random.default_rng(5)
    for sc in (case[3], case[4]):
        sc[r.random(sc.shape) < 0.2] *= -1
        sc[r.random(sc.shape) < 0.1] = 0
    case[4][r.random(case[4].shape) < 0.3] *= 500
    case[4][r.random(case[4].shape) < 0.3] *= 0.05
    q, kq, vq, ks, vs, tab, cu, lens = case
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = _run(case, 128 ** -0.5, err=err)
    want, bound = _reference(*case, 128 ** -0.5)
    # the bound's largest V scale counts by magnitude
    bound += lens.max() * 128 * 2.0 ** -25 * np.nanmax(np.abs(vs))
    assert int(err) == 0 and (np.abs(out.cpu().double().numpy() - want) <= bound).all()


def test_bad_data_is_flagged():
    case = _case(23, [30, 20, 1, 40], [100, 19, 60, 70], 16, 4, 16, "f16")
    q, kq, vq, ks, vs, tab, cu, lens = case
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = _run(case, 128 ** -0.5, err=err)
    assert int(err) == P.DEVERR["length"]                     # 20 rows, 19 keys
    want, bound = _reference(*case, 128 ** -0.5, skip=(1,))
    ok = np.r_[0:30, 50:91]
    assert (np.abs(out.cpu().double().numpy() - want) <= bound)[ok].all()
    lens[1] = 20
    tab[3, 2] = 1 << 20
    err.zero_()
    _run(case, 128 ** -0.5, err=err)
    assert int(err) == P.DEVERR["block"]


def test_nothing_to_do():
    case = _case(29, [0, 0], [5, 0], 16, 4, 16, "f16")
    assert _run(case, 1.0).shape == (0, 16, 128)
    q, kq, vq, ks, vs, tab, cu, lens = case
    out = P.attn_varlen_int8(q.cuda(), *[torch.from_numpy(x).cuda() for x in (kq, vq, ks, vs, tab[:0], cu[:1], lens[:0])], 0, 1.0)
    assert out.shape == (0, 16, 128)


def test_rows_behind_the_last_sequence_stay():
    """A padded step: query rows, outputs and tables past the sequences' own are neither read into results nor written."""
    q, kq, vq, ks, vs, tab, cu, lens = _case(43, [40, 1, 33], [40, 90, 200], 16, 4, 16, "f16")
    pad = torch.full((50, 16, 128), float("nan"), dtype=q.dtype)
    out = torch.full((124, 16, 128), 7.0, device="cuda")
    dev = [torch.from_numpy(x).cuda() for x in (kq, vq, ks, vs, tab, cu, lens)]
    P.attn_varlen_int8(torch.cat([q, pad]).cuda(), *dev, 40, 128 ** -0.5, out=out)
    _check((q, kq, vq, ks, vs, tab, cu, lens), 128 ** -0.5, got=out[:74])
    assert (out[74:] == 7.0).all()


def test_same_bits_every_time_and_replayed():
    case = _case(31, [257, 1, 66], [700, 90, 66], 32, 8, 32, "bf16")
    q, *rest = case
    dev = [torch.from_numpy(x).cuda() for x in rest]
    dq = q.cuda()
    out = torch.empty(324, 32, 128, device="cuda")
    ws = torch.empty(P.varlen_workspace_size(3, 32, 8, 128), dtype=torch.uint8, device="cuda")

    def step():
        P.attn_varlen_int8(dq, *dev, 257, 128 ** -0.5, out=out, workspace=ws)

    step()
    first = out.clone()
    graph = P.StepGraph(step)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)


def test_refusals():
    q, kq, vq, ks, vs, tab, cu, lens = [x.cuda() if isinstance(x, torch.Tensor) else torch.from_numpy(x).cuda()
                                        for x in _case(37, [30, 1], [100, 60], 16, 4, 16, "f16")]
    base = dict(q=q, kq=kq, vq=vq, k_scale=ks, v_scale=vs, block_tables=tab, cu_seqlens_q=cu, seq_lens=lens, max_q_len=30,
                scale=0.1)
    P.attn_varlen_int8(**base)
    odd = torch.zeros(31 * 16 * 128 + 4, dtype=torch.float16, device="cuda")[4:].view(31, 16, 128)
    for bad, kind in [(dict(q=q.float()), TypeError), (dict(q=q[:, :15]), ValueError), (dict(q=q[:, :, :64].contiguous()), ValueError),
                      (dict(q=odd), P.PkvError), (dict(cu_seqlens_q=cu[:2]), ValueError), (dict(cu_seqlens_q=cu.long()), TypeError),
                      (dict(seq_lens=lens[:1]), ValueError), (dict(block_tables=tab[:1]), ValueError),
                      (dict(k_scale=ks.half()), TypeError), (dict(kq=kq.cpu()), TypeError), (dict(out_dtype=torch.bfloat16), P.PkvError),
                      (dict(out=torch.empty(31, 16, 64, device="cuda")), ValueError),
                      (dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda")), P.PkvError),
                      (dict(max_q_len=-1), P.PkvError)]:
        with pytest.raises(kind):
            P.attn_varlen_int8(**{**base, **bad})


def test_an_int8_cache_from_prompt_to_eviction():
    """Chunks of a prompt written and attended over an int8 cache, decode steps that accumulate weights, a cut, more
    steps: every output against binary64 attention over the codes and scales the cache holds at that point."""
    hq, hkv, bs, d, budget = 16, 4, 32, 128, 96
    g = W.generator(91)
    a = P.BlockAllocator(64, bs)
    seqs = [a.create_sequence() for _ in range(3)]
    pools = [torch.zeros(64, bs, hkv, d, dtype=torch.int8, device="cuda") for _ in range(2)]
    pools += [torch.zeros(64, hkv, device="cuda") for _ in range(2)]
    mb = 8
    tables, lens = torch.empty(3, mb, dtype=torch.int32), torch.empty(3, dtype=torch.int32)
    weights = torch.zeros(3, hkv, mb * bs, device="cuda")
    scale = d ** -0.5

    def state():
        return [x.cpu().numpy() for x in pools] + [tables.numpy().copy()]

    def step(counts):
        slots, _ = a.append_tokens(seqs, counts)
        k, v = (W.normal(g, (len(slots), hkv, d), 1.0, "f16").cuda() for _ in range(2))
        P.write_kv_int8(k, v, torch.tensor(slots, dtype=torch.int64, device="cuda"), *pools)
        a.fill_tables(seqs, mb, tables, lens)
        q = W.normal(g, (sum(counts), hq, d), 1.0, "f16")
        cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        return q, cu, tables.cuda(), lens.cuda()

    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for counts in ([70, 33, 100], [60, 1, 28], [1, 90, 2]):
        q, cu, dt, dl = step(counts)
        out = P.attn_varlen_int8(q.cuda(), *pools, dt, torch.from_numpy(cu).cuda(), dl, max(counts), scale, err=err)
        want, bound = _reference(q, *state(), cu, lens.numpy(), scale)
        assert (np.abs(out.cpu().double().numpy() - want) <= bound).all()
    for i in range(20):
        q, cu, dt, dl = step([1, 1, 1])
        out = P.attn_decode_int8(q.cuda(), *pools, dt, dl, scale, key_weights=weights, err=err)
        want, bound = _reference(q, *state(), cu, lens.numpy(), scale)
        assert (np.abs(out.cpu().double().numpy() - want) <= bound).all()
        if i == 9:
            before, old = [x.clone() for x in pools], lens.clone()
            kept, new = P.evict_select(weights, dl, budget, sink=2, recent=16, err=err)
            P.evict_compact_int8(*pools, dt, dl, kept, key_weights=weights, err=err)
            for s, sid in enumerate(seqs):
                a.truncate(sid, min(budget, int(old[s])))
            assert new.tolist() == [budget] * 3
            # the kept rows' values moved, within half a step of their block's new scale
            for s in range(3):
                for h in range(hkv):
                    src, dst = kept[s, h].long(), torch.arange(budget, device="cuda")
                    tab = dt[s].long()
                    for x, y, sc, nsc in ((before[0], pools[0], before[2], pools[2]), (before[1], pools[1], before[3], pools[3])):
                        was = x[tab[src // bs], src % bs, h].double() * sc[tab[src // bs], h].double()[:, None]
                        now = y[tab[dst // bs], dst % bs, h].double() * nsc[tab[dst // bs], h].double()[:, None]
                        # half a step, and 2 2^-24 of up to 127 steps for the binary32 value and quotient
                        assert ((was - now).abs() <= nsc[tab[dst // bs], h].double()[:, None] * (0.5 + 2.0 ** -16)).all()
    assert int(err) == 0
