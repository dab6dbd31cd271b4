"""8-bit caches on the GPU against the float64 oracle (oracle/kv8_ref.py): append, read, dense
and sparse attention with accumulated weights, eviction, and runs of them together."""
import numpy as np
import pytest
import torch

import oracle
import token_level_sparse_fwht_b200 as ad
from kv8_helpers import D, Case, attention_oracle, check
from oracle import kv8_ref as ref

pytestmark = pytest.mark.gpu
FMTS = ["e4m3", "int8"]


def up(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def fine(ws):
    ad.check_workspace(ws)


# ------------------------------------------------------------------------- read
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("page", [0, 32])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_read_gives_the_values(fmt, page, dtype):
    c = Case(3, 2, 130, fmt, block=16, page=page, seed=1)
    cache = c.upload(ad)
    ws = ad.kv8_workspace()
    starts = [0, 7, 40]
    k, v = ad.kv8_read(cache, i32(starts), 77, ws, dtype=dtype)
    fine(ws)
    for got, want in zip((k, v), c.values()):
        for b, s in enumerate(starts):
            assert np.array_equal(got[b].double().cpu().numpy(), want[b, :, s:s + 77])


def test_read_every_byte_and_outside_positions():
    vals = ref.e4m3_values()
    k = torch.arange(256, dtype=torch.uint8).view(1, 1, 2, D).cuda()
    sc = torch.tensor([[[0.5, 4.0]]]).cuda()
    cache = ad.KV8Cache(k.view(torch.float8_e4m3fn), k.flip(-1).contiguous().view(torch.float8_e4m3fn),
                        sc, sc, 1)
    ws = ad.kv8_workspace()
    got, _ = ad.kv8_read(cache, 0, 2, ws, dtype=torch.float32)
    fine(ws)
    want = vals.reshape(2, D) * np.array([[0.5], [4.0]])
    assert np.array_equal(got[0, 0].double().cpu().numpy(), want, equal_nan=True)
    got, _ = ad.kv8_read(cache, -1, 4, ws)          # one row before, one behind: zeros, recorded
    assert (got[0, 0, [0, 3]] == 0).all() and not (got[0, 0, 1] == 0).all()
    with pytest.raises(ad.AdamasError):
        ad.check_workspace(ws)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("e", [-110, 95, 106])
def test_read_of_very_large_and_very_small_scales(fmt, e):
    c = Case(1, 2, 130, fmt, block=16, seed=2)
    c.ks, c.vs = c.ks * 2.0 ** e, c.vs * 2.0 ** e
    ws = ad.kv8_workspace()
    got = ad.kv8_read(c.upload(ad), 0, 130, ws, dtype=torch.float32)
    fine(ws)
    for g, want in zip(got, c.values()):
        assert np.abs(want).max() < 2.0 ** 127
        assert np.array_equal(g.double().cpu().numpy(), want[:, :, :130])


# ----------------------------------------------------------------------- append
def _append_case(fmt, dtype, block, page, B, Hkv, L, starts, counts, n, seed, layout="bhnd", codes=None):
    c = Case(B, Hkv, L, fmt, block=block, page=page, seed=seed, codes=codes is not None)
    cache = c.upload(ad)
    rng = np.random.default_rng(seed + 100)
    x = rng.standard_normal((2, B, Hkv, n, D)) * np.exp2(rng.integers(-6, 7, (2, B, Hkv, n, 1)))
    x = torch.from_numpy(x).to(dtype)
    for b in range(B):                              # rows past a sequence's count are never read
        x[:, b, :, counts[b]:] = float("nan")
    if layout == "bhnd":
        kn, vn = x[0].cuda(), x[1].cuda()
    else:                                           # slices of a token-major projection
        both = torch.cat([x[0], x[1]], 1).transpose(1, 2).contiguous().cuda()
        kn, vn = both.transpose(1, 2)[:, :Hkv], both.transpose(1, 2)[:, Hkv:]
    ws = ad.kv8_workspace()
    kw = {} if codes is None else codes
    ad.kv8_append(cache, kn, vn, i32(starts), ws, counts=i32(counts), **kw)
    fine(ws)
    k, ks, v, vs, cd = c.download(cache)
    xs = x.double().numpy()
    for b in range(B):
        for h in range(Hkv):
            for got, gs, st, sc, new in ((k, ks, c.k, c.ks, xs[0]), (v, vs, c.v, c.vs, xs[1])):
                want, wsc = ref.append(st[b, h], sc[b, h], new[b, h, :counts[b]], starts[b], fmt, block)
                assert np.array_equal(gs[b, h], wsc), (b, h)
                assert np.array_equal(got[b, h], want), (b, h)
    return c, cd, x


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block,page", [(1, 0), (2, 4), (4, 0), (8, 8), (16, 0), (64, 64), (32, 128),
                                        (128, 0), (256, 256)])
def test_append_matches_oracle(fmt, dtype, block, page):
    n = 150
    starts, counts = [0, 5, 63, 100, 257], [n, 1, 0, 37, 129]
    _append_case(fmt, dtype, block, page, 5, 2, 512, starts, counts, n, seed=block)


@pytest.mark.parametrize("fmt", FMTS)
def test_append_from_strided_projection(fmt):
    _append_case(fmt, torch.bfloat16, 16, 0, 2, 3, 256, [3, 200], [20, 56], 56, seed=5, layout="bnhd")


def test_append_token_by_token_equals_the_oracles_steps():
    """One token a time through three blocks: scales grow, earlier rows are rounded again."""
    fmt, block = "int8", 8
    c = Case(1, 2, 24, fmt, block=block, empty=True)
    cache = c.upload(ad)
    ws = ad.kv8_workspace()
    rng = np.random.default_rng(3)
    st = [[c.k[0, h] * 0, np.zeros(3)] for h in range(2)]
    for i in range(24):
        x = torch.from_numpy(rng.standard_normal((1, 2, 1, D)) * 2.0 ** (i % 8)).to(torch.bfloat16)
        ad.kv8_append(cache, x.cuda(), x.cuda(), i, ws)
        for h in range(2):
            st[h] = list(ref.append(*st[h], x[0, h].double().numpy(), i, fmt, block))
    fine(ws)
    k, ks, v, vs, _ = c.download(cache)
    for h in range(2):
        assert np.array_equal(k[0, h], st[h][0]) and np.array_equal(ks[0, h], st[h][1])
        assert np.array_equal(v[0, h], st[h][0]) and np.array_equal(vs[0, h], st[h][1])


@pytest.mark.parametrize("fmt", FMTS)
def test_append_extreme_values(fmt):
    """Zero rows, tiny and large magnitudes, magnitudes on the scale's border, and non-finite elements."""
    top = ref.FMAX[fmt]
    rows = np.zeros((8, D))
    rows[1, :4] = [1e-38, -2e-38, 1e-40, 0]
    rows[2] = np.linspace(-1, 1, D) * 1e30
    rows[3, 0], rows[3, 1] = top, -top                # exactly the largest: scale 1
    rows[4, 0] = np.nextafter(np.float32(top), np.float32(np.inf))   # just above: scale 2
    rows[5, :3] = [1.0, np.nan, 2.0]
    rows[6, :3] = [1.0, np.inf, -np.inf]
    rows[7] = np.arange(D) / 16 * (2.5 if fmt == "e4m3" else 0.5)    # ties
    x = torch.from_numpy(rows).float().view(1, 1, 8, D).cuda()
    c = Case(1, 1, 8, fmt, block=1)
    cache = c.upload(ad)
    ws = ad.kv8_workspace()
    ad.kv8_append(cache, x, x, 0, ws)
    fine(ws)
    k, ks, v, vs, _ = c.download(cache)
    for r in range(8):
        row = rows[r].astype(np.float32).astype(np.float64)
        with np.errstate(invalid="ignore"):
            want, sc = ref.append(np.zeros((1, D)), np.zeros(1), row[None], 0, fmt, 1)
        if fmt == "int8":
            want = np.nan_to_num(want, nan=0.0)
        assert ks[0, 0, r] == sc[0] == vs[0, 0, r], r
        assert np.array_equal(k[0, 0, r], want[0], equal_nan=True), r
    assert ks[0, 0, 0] == 2.0 ** -126 and ks[0, 0, 3] == 1.0 and ks[0, 0, 4] == 2.0


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("kw", [dict(t=1.01), dict(t=0.0), dict(ratio=0.5)])
def test_append_codes(page, kw):
    """The codes of the rows as given (not as quantised), only at the new positions."""
    starts, counts, n = [0, 11], [40, 29], 40
    c, codes, x = _append_case("e4m3", torch.bfloat16, 16, page, 2, 2, 64, starts, counts, n, seed=8,
                               codes=kw)
    for b in range(2):
        rows = x[0, b, :, :counts[b]].double().numpy()
        y = oracle.hadamard_rotate(rows)
        if "t" in kw:
            want, margin = oracle.bucketize(y, kw["t"]), oracle.threshold_margin(y, kw["t"])
        else:
            t = oracle.absmax_thresholds(rows, 0.5)
            want = oracle.bucketize_per_vector(y, t)
            margin = np.minimum(np.abs(np.abs(y) - np.asarray(t).reshape(*y.shape[:-1], 1)), np.abs(y))
        got = oracle.unpack_codes(codes[b, :, starts[b]:starts[b] + counts[b]])
        # fp32 transform: a coordinate within 1e-4 of its vector's scale of a threshold may differ
        near = margin < 1e-4 * np.maximum(1.0, np.abs(y).max(-1, keepdims=True))
        assert not ((got != want) & ~near).any()
        rest = np.ones(c.cap, bool)
        rest[starts[b]:starts[b] + counts[b]] = False
        assert (codes[b][:, rest] == 0).all()


def test_append_records_bad_positions_and_pages_and_writes_nothing_there():
    c = Case(4, 1, 64, "e4m3", block=16, page=16, seed=2)
    c.table[3, 1] = c.num_pages + 5                   # position 16.. of sequence 3 has no page
    table = c.table.copy()
    c.table[3, 1] = [p for p in range(c.num_pages) if p not in set(table.ravel())][0]
    cache = c.upload(ad)
    cache.block_table.copy_(torch.from_numpy(table))
    ws = ad.kv8_workspace()
    x = torch.ones((4, 1, 8, D), dtype=torch.bfloat16, device="cuda")
    before = [t.clone() for t in (cache.k.view(torch.uint8), cache.k_scale)]
    ad.kv8_append(cache, x, x, i32([60, -1, 3, 20]), ws, counts=i32([8, 8, 9, 8]))
    with pytest.raises(ad.AdamasError) as e:
        ad.check_workspace(ws)
    assert e.value.status == ad.ERR_INVALID_ARG
    assert torch.equal(cache.k.view(torch.uint8), before[0]) and torch.equal(cache.k_scale, before[1])


# ------------------------------------------------------------------- dense attention
def _dense(c, cache, q, lens, weights=False, inplace=True, ws=None):
    Hq = q.shape[1]
    if ws is None:
        ws = ad.kv8_attention_workspace(c.B, Hq, c.Hkv, cache.Lmax, weights=weights)
    if not weights:
        out = ad.kv8_attention(q, cache, lens, ws)
        fine(ws)
        return out, None, None
    w0 = torch.rand((c.B, c.Hkv, cache.Lmax), device="cuda")
    w = w0.clone()
    if inplace:
        out = ad.kv8_attention(q, cache, lens, ws, weights=w)
    else:
        out = ad.kv8_attention(q, cache, lens, ws, weights=w0.clone(), weights_out=w)
    fine(ws)
    return out, w0, w


def _check_dense(c, cache, q, lens, weights=False, inplace=True, ws=None):
    want, tol, ww, wtol = attention_oracle(q.double().cpu().numpy(), c, lambda b, h: np.arange(lens[b]))
    out, w0, w = _dense(c, cache, q, i32(lens), weights, inplace, ws)
    check(out, want, tol, "out")
    if weights:
        base = np.zeros((c.B, c.Hkv, cache.Lmax))
        n = min(c.cap, cache.Lmax)
        base[..., :n], t = ww[..., :n], np.zeros_like(base)
        t[..., :n] = wtol[..., :n]
        w0 = w0.double().cpu().numpy()
        check(w, w0 + base, t + (w0 + base) * 2.0 ** -23, "weights")
        for b in range(c.B):                          # behind a sequence: left as they were
            assert np.array_equal(w[b, :, lens[b]:].double().cpu().numpy(), w0[b, :, lens[b]:])
    return out


def _q(B, Hq, dtype, seed=0, amp=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((B, Hq, D), generator=g) * amp).to(dtype).cuda()


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dense_head_groups(G, fmt, dtype):
    c = Case(2, 2, 300, fmt, block=16, seed=G)
    _check_dense(c, c.upload(ad), _q(2, 2 * G, dtype, G), [300, 137], weights=True)


@pytest.mark.parametrize("block,page", [(1, 0), (1, 1), (2, 2), (4, 16), (8, 0), (16, 64), (64, 0),
                                        (128, 128), (256, 0)])
@pytest.mark.parametrize("fmt", FMTS)
def test_dense_blocks_and_pages(block, page, fmt):
    c = Case(5, 2, 400, fmt, block=block, page=page, seed=block + page)
    lens = [400, 0, 1, 255, 17]
    _check_dense(c, c.upload(ad), _q(5, 8, torch.bfloat16, 1), lens, weights=True, inplace=False)


@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 127, 128, 129, 1000, 4097])
def test_dense_lengths(L):
    c = Case(1, 2, L, "e4m3", block=8, seed=L)
    _check_dense(c, c.upload(ad), _q(1, 8, torch.bfloat16, L), [L])


def test_dense_one_long_sequence_over_all_ctas():
    c = Case(1, 1, 70001, "e4m3", block=64, seed=4)
    _check_dense(c, c.upload(ad), _q(1, 4, torch.float32, 3), [70001], weights=True)


def test_dense_many_short_sequences():
    rng = np.random.default_rng(0)
    lens = [int(x) for x in rng.integers(0, 200, 150)]
    c = Case(150, 2, 200, "int8", block=8, page=8, seed=6)
    _check_dense(c, c.upload(ad, max_seq_len=200), _q(150, 16, torch.bfloat16, 3), lens, weights=True)


@pytest.mark.parametrize("G,at", [(1, 0), (3, 17), (8, 39)])
def test_dense_one_long_sequence_among_short_ones(G, at):
    lens = [int(x) for x in np.random.default_rng(G).integers(0, 60, 40)]
    lens[at] = 4000
    c = Case(40, 1, 4000, "int8", block=16, seed=G)
    _check_dense(c, c.upload(ad), _q(40, G, torch.bfloat16, 7), lens, weights=True)


@pytest.mark.parametrize("L", [128 * 8, 128 * 8 + 1, 128 * 9 + 1, 128 * 10])
def test_dense_units_of_few_and_of_many_parts(L):
    c = Case(1, 3, L, "e4m3", block=64, seed=8)
    _check_dense(c, c.upload(ad), _q(1, 24, torch.bfloat16, 7), [L], weights=True)


def test_dense_all_sequences_empty():
    c = Case(3, 2, 64, "e4m3")
    out = _check_dense(c, c.upload(ad), _q(3, 4, torch.bfloat16), [0, 0, 0], weights=True)
    assert (out == 0).all()


def test_dense_without_lengths_covers_the_cache():
    c = Case(2, 2, 256, "e4m3", block=64, seed=9)
    cache, q = c.upload(ad), _q(2, 8, torch.bfloat16)
    ws = ad.kv8_attention_workspace(2, 8, 2, cache.Lmax)
    a = ad.kv8_attention(q, cache, None, ws)
    b = ad.kv8_attention(q, cache, i32([256, 256]), ws)
    fine(ws)
    assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", FMTS)
def test_dense_scales_of_another_quantiser_and_extreme_spread(fmt):
    c = Case(1, 2, 320, fmt, block=16, seed=12, pow2=False)
    _check_dense(c, c.upload(ad), _q(1, 8, torch.float32, 5), [311], weights=True)
    # V scales from 2^-90 to 2^60 between blocks, K at 2^40, q at 2^-40
    c = Case(1, 1, 64, fmt, block=16, seed=13, amp=1.0, spread=0)
    c.vs *= np.array([2.0 ** -90, 1.0, 2.0 ** 60, 2.0 ** -126])
    c.ks *= 2.0 ** 40
    _check_dense(c, c.upload(ad), _q(1, 2, torch.float32, 6, amp=2.0 ** -40), [64])
    c.vs = np.full_like(c.vs, 2.0 ** -120)            # every value tiny
    _check_dense(c, c.upload(ad), _q(1, 2, torch.float32, 6, amp=2.0 ** -40), [64])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("e", [-100, 100])
@pytest.mark.parametrize("block", [4, 16])
def test_dense_very_large_and_very_small_values(fmt, e, block):
    c = Case(2, 2, 300, fmt, block=block, seed=3)
    c.vs = c.vs * 2.0 ** e
    _check_dense(c, c.upload(ad), _q(2, 8, torch.bfloat16, 5), [300, 41], weights=True)


def test_dense_dead_rows_may_hold_anything():
    """Bytes and scales behind a sequence's end: NaN bytes, NaN and infinite scales."""
    c = Case(2, 2, 96, "e4m3", block=16, seed=3)
    cache, q = c.upload(ad), _q(2, 8, torch.bfloat16, 2)
    for t in (cache.k, cache.v):
        t.view(torch.uint8)[0, :, 50:] = 0x7F
        t.view(torch.uint8)[1, :, 0:] = 0xFF
    for t in (cache.k_scale, cache.v_scale):
        t[0, :, 4:] = float("nan")
        t[1] = float("inf")
    _check_dense(c, cache, q, [50, 0], weights=True)


def test_dense_nan_key_shows():
    c = Case(1, 1, 40, "e4m3", block=8, seed=3)
    cache, q = c.upload(ad), _q(1, 2, torch.bfloat16, 2)
    cache.k.view(torch.uint8)[0, 0, 7, 5] = 0x7F
    ws = ad.kv8_attention_workspace(1, 2, 1, cache.Lmax)
    assert torch.isnan(ad.kv8_attention(q, cache, i32([40]), ws)).all()
    assert torch.isfinite(ad.kv8_attention(q, cache, i32([7]), ws)).all()
    fine(ws)


def test_dense_sharp_softmax_and_equal_keys():
    """One dominating key far from the rest (scores of hundreds), and identical keys."""
    c = Case(1, 1, 512, "e4m3", block=16, seed=21, spread=0)
    q = _q(1, 4, torch.bfloat16, 2, amp=30.0)
    _check_dense(c, c.upload(ad), q, [512], weights=True)
    c.k[:] = c.k[:, :, :1]
    c.ks[:] = 1.0
    _check_dense(c, c.upload(ad), q, [500], weights=True)


def test_dense_bad_lengths_and_pages_are_recorded():
    c = Case(2, 1, 64, "e4m3", block=16, page=16, seed=2)
    cache, q = c.upload(ad), _q(2, 2, torch.bfloat16)
    ws = ad.kv8_attention_workspace(2, 2, 1, cache.Lmax, weights=True)
    out = ad.kv8_attention(q, cache, i32([65, -3]), ws)
    with pytest.raises(ad.AdamasError):
        ad.check_workspace(ws)
    want, tol, _, _ = attention_oracle(q.double().cpu().numpy(), c, lambda b, h: np.arange([64, 0][b]))
    check(out, want, tol, "clamped lengths")
    ad.init_workspace(ws)
    cache.block_table[0, 1] = -1                      # positions 16..31 drop out
    cache.block_table[1, 0] = c.num_pages
    w = torch.zeros((2, 1, cache.Lmax), device="cuda")
    out = ad.kv8_attention(q, cache, i32([40, 16]), ws, weights=w)
    with pytest.raises(ad.AdamasError):
        ad.check_workspace(ws)
    pos = [np.r_[0:16, 32:40], np.arange(0)]
    want, tol, ww, wtol = attention_oracle(q.double().cpu().numpy(), c, lambda b, h: pos[b])
    check(out, want, tol, "missing pages")
    check(w, ww, wtol, "weights")


# ------------------------------------------------------------------ sparse attention
def _check_sparse(c, cache, q, idx, shared, weights=True, inplace=True):
    Hq = q.shape[1]
    G = Hq // c.Hkv
    lists = lambda b, h: idx[b, h // G if shared else h][idx[b, h // G if shared else h] >= 0]  # noqa: E731
    want, tol, ww, wtol = attention_oracle(q.double().cpu().numpy(), c, lists)
    ws = ad.kv8_sparse_attention_workspace(c.B, Hq, c.Hkv, idx.shape[-1], shared=shared, weights=weights)
    kw = {}
    w0 = torch.rand((c.B, c.Hkv, cache.Lmax), device="cuda")
    w = w0.clone()
    if weights:
        kw = dict(weights=w) if inplace else dict(weights=w0, weights_out=w.fill_(7.0))
    out = ad.kv8_sparse_attention(q, cache, up(idx.astype(np.int32)), ws, shared=shared, **kw)
    fine(ws)
    check(out, want, tol, "out")
    if weights:
        n = min(c.cap, cache.Lmax)
        base, t = np.zeros(w0.shape), np.zeros(w0.shape)
        base[..., :n], t[..., :n] = ww[..., :n], wtol[..., :n]
        base += w0.double().cpu().numpy()
        check(w, base, t + base * 2.0 ** -22, "weights")
    return out


def _lists(rng, B, rows, L, k, drop=0.0):
    idx = np.stack([np.stack([np.sort(rng.choice(L, k, replace=False)) for _ in range(rows)])
                    for _ in range(B)])
    return np.where(rng.random(idx.shape) < drop, -1, idx)


@pytest.mark.parametrize("G", [1, 3, 4, 8])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("fmt", FMTS)
def test_sparse_lists(G, shared, fmt):
    c = Case(2, 2, 500, fmt, block=16, page=32 if G == 4 else 0, seed=G)
    rng = np.random.default_rng(G)
    idx = _lists(rng, 2, 2 if shared else 2 * G, 500, 77)
    _check_sparse(c, c.upload(ad), _q(2, 2 * G, torch.bfloat16, G), idx, shared, inplace=G != 3)


@pytest.mark.parametrize("k", [1, 15, 128, 129, 400])
def test_sparse_list_lengths(k):
    c = Case(1, 2, 400, "e4m3", block=64, seed=k)
    _check_sparse(c, c.upload(ad), _q(1, 4, torch.float32, k), _lists(np.random.default_rng(k), 1, 4, 400, k),
                  False)


@pytest.mark.parametrize("shared", [False, True])
def test_sparse_gaps_repeats_and_any_order(shared):
    c = Case(2, 2, 300, "int8", block=8, seed=5)
    rng = np.random.default_rng(1)
    R = 2 if shared else 4
    idx = _lists(rng, 2, R, 300, 200, drop=0.3)
    idx[0, 0] = rng.permutation(idx[0, 0])
    idx[0, 1] = -1                                    # nothing left
    idx[1, 0, :150] = -1                              # whole tiles of gaps
    idx[1, 1] = 17                                    # one position, 200 times
    idx[1, 1, 5] = 299
    _check_sparse(c, c.upload(ad), _q(2, 4, torch.bfloat16, 2), idx, shared)


def test_sparse_over_several_weight_slices():
    c = Case(1, 1, 20000, "e4m3", block=64, seed=7)
    idx = _lists(np.random.default_rng(2), 1, 4, 20000, 1500)
    _check_sparse(c, c.upload(ad), _q(1, 4, torch.bfloat16, 3), idx, False, inplace=False)


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("inplace", [False, True])
def test_sparse_weights_of_many_long_sequences(shared, inplace):
    """Enough slices to fill the device are taken wide: the sums of 76 sequences at once are those
    of 19 at a time, bit for bit (lists of one step: the attention's own results do not differ)."""
    B, L, Hq, k = 76, 8300, 4, 100
    g = torch.Generator(device="cuda").manual_seed(3)
    kv = [torch.randint(-127, 128, (B, 2, L + 20, D), generator=g, device="cuda").to(torch.int8)
          for _ in range(2)]
    sc = torch.exp2(torch.randint(-9, -6, (B, 2, (L + 20) // 16), generator=g, device="cuda").float())
    q = torch.randn((B, Hq, D), generator=g, device="cuda").bfloat16()
    idx = torch.from_numpy(_lists(np.random.default_rng(4), B, 2 if shared else Hq, L, k, drop=0.1)).int().cuda()
    w0 = torch.rand((B, 2, L + 20), generator=g, device="cuda")

    def run(s):
        cache = ad.KV8Cache(kv[0][s], kv[1][s], sc[s], sc[s], 16)
        n = q[s].shape[0]
        ws = ad.kv8_sparse_attention_workspace(n, Hq, 2, k, shared=shared, weights=True)
        w, start = torch.full_like(w0[s], 5.0), w0[s].clone()
        out = ad.kv8_sparse_attention(q[s], cache, idx[s], ws, shared=shared, weights=start,
                                      **({} if inplace else dict(weights_out=w)))
        fine(ws)
        return out, start if inplace else w

    out, w = run(slice(0, B))
    for b in range(0, B, 19):
        o, ww = run(slice(b, b + 19))
        assert torch.equal(out[b:b + 19], o) and torch.equal(w[b:b + 19], ww)
    heads = (idx >= 0).any(-1).double().sum(1) * (Hq // 2 if shared else 1)
    # each weight is off by a few 2^-24 of itself, and the running sum (below 5) rounds once per place
    assert torch.allclose((w.double() - w0.double()).sum((1, 2)), heads, rtol=0, atol=2 * Hq * k * 2.0 ** -22)


def test_sparse_positions_out_of_range_are_recorded():
    c = Case(1, 1, 64, "e4m3", block=16, seed=7)
    cache, q = c.upload(ad), _q(1, 1, torch.bfloat16)
    ws = ad.kv8_sparse_attention_workspace(1, 1, 1, 3, weights=True)
    w = torch.zeros((1, 1, 64), device="cuda")
    out = ad.kv8_sparse_attention(q, cache, i32([[[3, 64, 2 ** 31 - 1]]]), ws, weights=w)
    with pytest.raises(ad.AdamasError):
        ad.check_workspace(ws)
    K, V = c.values()
    assert np.allclose(out.cpu().double().numpy()[0, 0], V[0, 0, 3], rtol=1e-6)
    assert float(w[0, 0, 3]) == pytest.approx(1.0, abs=1e-6) and float(w.sum()) == float(w[0, 0, 3])


def test_sparse_of_every_position_is_dense():
    c = Case(1, 2, 700, "e4m3", block=64, seed=11)
    cache, q = c.upload(ad), _q(1, 8, torch.bfloat16, 4)
    idx = np.tile(np.arange(700), (1, 2, 1))
    a = _check_sparse(c, cache, q, idx, True)
    ws = ad.kv8_attention_workspace(1, 8, 2, cache.Lmax)
    assert torch.equal(a, ad.kv8_attention(q, cache, i32([700]), ws))


# ------------------------------------------------------------------------ eviction
def _weights(rng, B, Hkv, L, ties=True):
    w = np.exp(3 * rng.standard_normal((B, Hkv, L)) - 4).astype(np.float32)
    if ties:
        w[rng.random(w.shape) < 0.5] = 0.0
        w[rng.random(w.shape) < 0.2] = 0.125
    return w


SELECT = [(100, 40, 2, 8), (100, 100, 0, 0), (100, 99, 0, 99), (100, 10, 10, 0), (100, 1, 0, 0),
          (1, 1, 0, 0), (5000, 1234, 4, 100), (5000, 4999, 0, 0), (33000, 8000, 1, 1000)]


@pytest.mark.parametrize("L,budget,sink,recent", SELECT)
def test_evict_select_matches_oracle(L, budget, sink, recent):
    rng = np.random.default_rng(L + budget)
    B, Hkv = 3, 2
    w = _weights(rng, B, Hkv, L)
    w[0, 0, rng.integers(0, L, 5)] = np.nan
    w[1, 1] *= -1                                     # negative, and -0 next to 0
    w[1, 0, : L // 2] = 0.5                           # one long tie
    lens = [L, max(1, L // 2), 0]
    ws = ad.kv8_workspace()
    wt, out = up(w), torch.full((B, Hkv, L + 3), 9.0, device="cuda")
    keep = ad.evict_select(wt, i32(lens), budget, ws, sink=sink, recent=recent, weights_out=out)
    fine(ws)
    keep, out = keep.cpu().numpy(), out.cpu().numpy()
    inplace = up(w)
    ad.evict_select(inplace, i32(lens), budget, ws, sink=sink, recent=recent, weights_out=inplace)
    inplace = inplace.cpu().numpy()
    for b in range(B):
        for h in range(Hkv):
            want = ref.evict_select(w[b, h], lens[b], budget, sink, recent)
            n = len(want)
            assert np.array_equal(keep[b, h, :n], want), (b, h)
            assert (keep[b, h, n:] == -1).all()
            assert np.array_equal(out[b, h, :n], w[b, h, want], equal_nan=True)
            assert (out[b, h, n:lens[b]] == 0).all() and (out[b, h, max(n, lens[b]):] == 9).all()
            assert np.array_equal(inplace[b, h, :n], w[b, h, want], equal_nan=True)
            assert (inplace[b, h, n:lens[b]] == 0).all()
            assert np.array_equal(inplace[b, h, lens[b]:], w[b, h, lens[b]:], equal_nan=True)


def test_evict_select_many_units_and_a_long_one():
    rng = np.random.default_rng(9)
    for B, Hkv, L, budget in ((40, 8, 700, 333), (1, 1, 300000, 20000)):
        w = _weights(rng, B, Hkv, L)
        ws = ad.kv8_workspace()
        keep = ad.evict_select(up(w), i32([L] * B), budget, ws, recent=50).cpu().numpy()
        fine(ws)
        for b in range(0, B, 7):
            for h in range(Hkv):
                assert np.array_equal(keep[b, h], ref.evict_select(w[b, h], L, budget, 0, 50))


def _check_evict(c, lens, budget, sink, recent, in_place, dst_block=None, seed=0):
    rng = np.random.default_rng(seed)
    if c.codes is not None:
        c.codes[:] = rng.integers(0, 256, c.codes.shape, dtype=np.uint8)
    cache = c.upload(ad)
    w = _weights(rng, c.B, c.Hkv, cache.Lmax)
    ws = ad.kv8_workspace()
    wt, lt = up(w), i32(lens)
    d, dst, kw = c, None, {}
    if not in_place:
        d = Case(c.B, c.Hkv, budget, c.fmt, block=dst_block or c.block, page=c.page, seed=seed + 1,
                 codes=c.codes is not None)
        dst = d.upload(ad)
        kw = dict(dst=dst)
    before = d.download(dst or cache)
    keep, new_lens = ad.kv8_evict(cache, wt, lt, budget, ws, sink=sink, recent=recent, **kw)
    fine(ws)
    got = d.download(dst or cache)
    assert new_lens.tolist() == [min(x, budget) for x in lens]
    vals = c.values()
    for b in range(c.B):
        for h in range(c.Hkv):
            sel = ref.evict_select(w[b, h], lens[b], budget, sink, recent)
            n = len(sel)
            assert np.array_equal(keep[b, h, :n].cpu().numpy(), sel)
            for i in (0, 2):
                stored, scale = ref.requantise(vals[i // 2][b, h, sel], c.fmt, d.block)
                have = got[i][b, h, :n] * got[i + 1][b, h].repeat(d.block)[:n, None]
                assert np.array_equal(have, stored * scale.repeat(d.block)[:n, None]), (b, h, i)
                assert np.array_equal(got[i][b, h, n:], before[i][b, h, n:])   # rows behind
            if c.codes is not None:
                assert np.array_equal(got[4][b, h, :n], c.codes[b, h, sel])
                assert np.array_equal(got[4][b, h, n:], before[4][b, h, n:])
    return cache, wt, lt


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("block,page", [(1, 0), (4, 8), (16, 0), (16, 32), (64, 64), (256, 0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_matches_oracle(fmt, block, page, in_place):
    c = Case(4, 2, 900, fmt, block=block, page=page, seed=block, codes=True, spread=5)
    _check_evict(c, [900, 300, 0, 451], 450, 3, 40, in_place)


def test_evict_in_place_over_many_rounds():
    c = Case(1, 2, 9000, "e4m3", block=16, seed=2, codes=True)
    _check_evict(c, [9000], 7777, 0, 100, True)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("block,page", [(16, 0), (8, 16), (256, 0)])
def test_evict_of_many_units_into_another_cache(fmt, block, page):
    """Enough chunks that a CTA takes several: selection, codes, sums and lengths are those of the move
    in place, values those of the definition (in place a block whose rows all stay keeps its
    bytes; requantised, a block that holds -128 goes to twice its scale and odd bytes round)."""
    B, H, budget = 32, 8, 1024
    L = budget + 256
    g = torch.Generator(device="cuda").manual_seed(block)
    rand = lambda *s: torch.randint(0, 256, s, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    lead = (B, H, L) if page == 0 else (B * L // page, H, page)

    def cache(k, v, ks, vs, codes, table):
        dt = torch.int8 if fmt == "int8" else torch.float8_e4m3fn
        return ad.KV8Cache(k.view(dt), v.view(dt), ks, vs, block, codes=codes, block_table=table)

    rows = [rand(*lead, D) for _ in range(2)]
    if fmt == "e4m3":
        rows = [torch.where((x & 127) == 127, x & 128, x) for x in rows]           # no NaN
    scales = [torch.exp2(torch.randint(-6, 6, (*lead[:2], lead[2] // block), generator=g, device="cuda").float())
              for _ in range(2)]
    table = None if page == 0 else torch.randperm(lead[0], generator=g, device="cuda").view(B, -1).int()
    parts = [*rows, *scales, rand(*lead, 32)]
    w = torch.rand((B, H, L), generator=g, device="cuda")
    lens = torch.randint(0, L + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    lens[0] = L
    src, there = (cache(*(x.clone() for x in parts), table) for _ in range(2))
    dst = cache(*(torch.zeros_like(x) for x in parts), table)
    olds = ad.kv8_read(src, 0, L, ad.kv8_workspace(), dtype=torch.float32)
    ws, out = ad.kv8_workspace(), torch.full_like(w, 7.0)
    keep, n = ad.kv8_evict(src, w, lens, budget, ws, sink=3, recent=50, dst=dst, weights_out=out)
    keep2, n2 = ad.kv8_evict(there, w, lens, budget, ws, sink=3, recent=50)
    fine(ws)
    assert torch.equal(keep, keep2) and torch.equal(n, n2)
    live = torch.arange(budget, device="cuda") < n[:, None, None]
    top = 448.0 if fmt == "e4m3" else 127.0
    for got, old in zip(ad.kv8_read(dst, 0, budget, ws, dtype=torch.float32), olds):
        v = old.gather(2, keep.clamp(min=0).long()[..., None].expand(-1, -1, -1, D)).double()
        v = v.masked_fill(~live[..., None], 0).view(B, H, budget // block, block, D)
        m, e = torch.frexp(v.abs().amax((-1, -2), keepdim=True) / top)
        scale = torch.exp2((e - (m == 0.5).int()).double().clamp(min=-126))
        x = (v / scale).float()
        x = x.round() if fmt == "int8" else x.to(torch.float8_e4m3fn).float()
        want = (x.double() * scale).view(B, H, budget, D)
        assert torch.equal(got.masked_fill(~live[..., None], 0).double(), want)
    by_position = lambda c: c.codes if page == 0 else c.codes[table.long()].transpose(1, 2).reshape(B, H, L, 32)  # noqa: E731
    a, b = by_position(dst)[:, :, :budget], by_position(there)[:, :, :budget]
    assert torch.equal(a * live[..., None], b * live[..., None]) and not (a * ~live[..., None]).any()
    assert torch.equal(out[:, :, :budget].masked_fill(~live, 0), w[:, :, :budget].masked_fill(~live, 0))


def test_evict_into_another_block_size():
    c = Case(2, 2, 500, "int8", block=8, seed=2, spread=6)
    _check_evict(c, [500, 77], 300, 0, 10, False, dst_block=32)


def test_evict_keeps_a_cache_within_budget_as_it_is():
    c = Case(2, 2, 128, "e4m3", block=16, seed=2, codes=True, pow2=False)
    cache = c.upload(ad)
    before = [t.clone() for t in (cache.k.view(torch.uint8), cache.k_scale, cache.v.view(torch.uint8),
                                  cache.v_scale)]
    w = torch.rand((2, 2, 128), device="cuda")
    w0, lens, ws = w.clone(), i32([128, 50]), ad.kv8_workspace()
    keep, _ = ad.kv8_evict(cache, w, lens, 128, ws, recent=5)
    fine(ws)
    after = (cache.k.view(torch.uint8), cache.k_scale, cache.v.view(torch.uint8), cache.v_scale)
    assert all(torch.equal(a, b) for a, b in zip(after, before)) and torch.equal(w, w0)
    assert lens.tolist() == [128, 50] and keep[1, 0, 49:51].tolist() == [49, -1]


@pytest.mark.parametrize("dtype,width", [(torch.bfloat16, D), (torch.float32, D), (torch.uint8, 32)])
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact_rows(dtype, width, page, in_place):
    rng = np.random.default_rng(4)
    B, Hkv, L, budget = 2, 3, 4000, 2600
    x = torch.from_numpy(rng.integers(0, 100, (B, Hkv, L, width))).to(dtype)
    w, lens = _weights(rng, B, Hkv, L), [L, 700]
    src, table = x, None
    if page:
        nb = L // page
        table = rng.permutation(B * nb).reshape(B, nb).astype(np.int32)
        src = torch.empty((B * nb, Hkv, page, width), dtype=dtype)
        for b in range(B):
            src[torch.from_numpy(table[b]).long()] = x[b].view(Hkv, nb, page, width).transpose(0, 1)
    src = src.cuda()
    dst = src if in_place else torch.zeros_like(src)
    before = dst.clone()
    ws = ad.kv8_workspace()
    keep = ad.evict_select(up(w), i32(lens), budget, ws, sink=2, recent=100)
    ad.compact_rows(src, keep, i32(lens), ws, dst=dst, block_table=None if table is None else up(table))
    fine(ws)

    def seq(t):
        if table is None:
            return t.cpu()
        return torch.stack([t.cpu()[torch.from_numpy(table[b]).long()].transpose(0, 1).reshape(Hkv, L, width)
                            for b in range(B)])
    got, before = seq(dst), seq(before)
    for b in range(B):
        for h in range(Hkv):
            sel = torch.from_numpy(ref.evict_select(w[b, h], lens[b], budget, 2, 100))
            assert torch.equal(got[b, h, :len(sel)], x[b, h, sel])
            assert torch.equal(got[b, h, len(sel):], before[b, h, len(sel):])


# ------------------------------------------------------------------- together
def test_serving_run_with_selection_and_eviction():
    """A prompt enters the cache with its codes; decode steps select by codes, attend over the
    selected 8-bit rows and sum weights; the cache is evicted and decoding goes on, then one dense
    step.  Every step against the oracle on the cache's own values."""
    B, Hkv, Hq, n, t, kk = 2, 2, 8, 300, 0.8, 48
    rng = np.random.default_rng(0)
    cache = ad.kv8_cache(B, Hkv, 400, block_size=16, codes=True)
    ws = ad.kv8_sparse_attention_workspace(B, Hq, Hkv, kk, weights=True)
    dws = ad.kv8_attention_workspace(B, Hq, Hkv, cache.Lmax, weights=True)
    sel_ws = ad.decode_workspace(B, Hq, Hkv, cache.Lmax, kk)
    w = torch.zeros((B, Hkv, cache.Lmax), device="cuda")
    lens = i32([300, 211])
    x = torch.from_numpy(rng.standard_normal((2, B, Hkv, n, D))).to(torch.bfloat16).cuda()
    ad.kv8_append(cache, x[0], x[1], 0, ws, counts=lens, t=t)

    def values():
        kv = [v.double().cpu().numpy() for v in ad.kv8_read(cache, 0, cache.Lmax, ws, torch.float32)]
        return *kv, cache.v_scale.double().cpu().numpy().repeat(16, 2)

    for step in range(4):
        x = torch.from_numpy(rng.standard_normal((2, B, Hkv, 1, D))).to(torch.bfloat16).cuda()
        ad.kv8_append(cache, x[0], x[1], lens, ws, t=t)
        lens += 1
        q = _q(B, Hq, torch.bfloat16, step)
        # selection over the codes, each sequence over its own length (per-head lists, -1 padded)
        idx = torch.full((B, Hq, kk), -1, dtype=torch.int32, device="cuda")
        qc = ad.encode_queries(q, t)
        for b in range(B):
            one = ad.select_topk(qc[b:b + 1].contiguous(), cache.codes[b:b + 1].contiguous(),
                                 int(lens[b]), kk, sel_ws)
            idx[b, :, :one.shape[-1]] = one[0]
        K, V, C = values()
        w0 = w.clone()
        out = ad.kv8_sparse_attention(q, cache, idx, ws, weights=w)
        ids = idx.cpu().numpy()
        want, tol, ww, wtol = attention_oracle(q.double().cpu().numpy(), (K, V, C),
                                               lambda b, h: ids[b, h][ids[b, h] >= 0])
        check(out, want, tol, f"step {step}")
        base = w0.double().cpu().numpy() + ww
        check(w, base, wtol + base * 2.0 ** -22, f"weights {step}")
        if step == 1:
            wn, ln, cn = w.cpu().numpy(), lens.tolist(), cache.codes.cpu().numpy()
            keep, _ = ad.kv8_evict(cache, w, lens, 220, ws, sink=4, recent=32)
            assert lens.tolist() == [220, 213]
            K2, V2, _ = values()
            for b in range(B):
                for h in range(Hkv):
                    s = ref.evict_select(wn[b, h], ln[b], 220, 4, 32)
                    assert np.array_equal(keep[b, h, :len(s)].cpu().numpy(), s)
                    for new, old in ((K2, K), (V2, V)):
                        st, sc = ref.requantise(old[b, h, s], "e4m3", 16)
                        assert np.array_equal(new[b, h, :len(s)], st * sc.repeat(16)[:len(s), None])
                    assert np.array_equal(cache.codes[b, h, :len(s)].cpu().numpy(), cn[b, h, s])
    q = _q(B, Hq, torch.float32, 77)
    out = ad.kv8_attention(q, cache, lens, dws, weights=w)
    ln = lens.tolist()
    want, tol, _, _ = attention_oracle(q.double().cpu().numpy(), values(), lambda b, h: np.arange(ln[b]))
    check(out, want, tol, "dense")
    for x in (ws, dws, sel_ws):
        fine(x)


def test_prepared_calls_in_a_graph_replay_with_new_data():
    c = Case(2, 2, 640, "e4m3", block=16, seed=3)
    cache, q = c.upload(ad), _q(2, 8, torch.bfloat16)
    lens = i32([0, 0])
    ws = ad.kv8_attention_workspace(2, 8, 2, cache.Lmax, weights=True)
    out = torch.empty((2, 8, D), device="cuda")
    w0 = torch.zeros((2, 2, cache.Lmax), device="cuda")
    w = torch.zeros_like(w0)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        ad.PreparedKV8Attention(q, cache, lens, ws, out, weights=w0, weights_out=w)()
    for n in ([640, 3], [200, 0], [1, 639]):
        lens.copy_(i32(n))
        q.copy_(_q(2, 8, torch.bfloat16, n[0]))
        graph.replay()
        torch.cuda.synchronize()
        eager = ad.kv8_attention(q, cache, lens, ad.kv8_attention_workspace(2, 8, 2, cache.Lmax))
        assert torch.equal(out, eager)
        _, _, ww, wtol = attention_oracle(q.double().cpu().numpy(), c, lambda b, h: np.arange(n[b]))
        for b in range(2):
            check(w[b, :, :n[b]], ww[b, :, :n[b]], wtol[b, :, :n[b]], "weights")
    fine(ws)


def test_two_streams_with_their_own_workspaces():
    cs = [Case(1, 2, 3000, "e4m3", block=16, seed=s) for s in (1, 2)]
    caches, qs = [c.upload(ad) for c in cs], [_q(1, 8, torch.bfloat16, s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for cache, q, s in zip(caches, qs, streams):
            ws = ad.kv8_attention_workspace(1, 8, 2, cache.Lmax, stream=s)
            outs.append(ad.kv8_attention(q, cache, None, ws, stream=s))
    torch.cuda.synchronize()
    for i, (c, q) in enumerate(zip(cs, qs)):
        want, tol, _, _ = attention_oracle(q.double().cpu().numpy(), c, lambda b, h: np.arange(c.cap))
        for o in outs[i::2]:
            check(o, want, tol, "out")


def test_same_call_twice_is_bitwise_the_same():
    c = Case(3, 2, 5000, "e4m3", block=16, seed=3)
    cache, q = c.upload(ad), _q(3, 8, torch.bfloat16)
    ws = ad.kv8_attention_workspace(3, 8, 2, cache.Lmax, weights=True)
    got = []
    for _ in range(3):
        w = torch.zeros((3, 2, cache.Lmax), device="cuda")
        got.append((ad.kv8_attention(q, cache, i32([5000, 77, 4000]), ws, weights=w), w))
    fine(ws)
    for o, w in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(w, got[0][1])


def test_rows_beyond_four_gigabytes():
    """Row offsets past 2^32 bytes: append, read, sparse and (over pages) dense attention, eviction's move
    at the far end of a cache of 40 million rows."""
    rows, L = 40_000_000, 20_000_000
    free, _ = torch.cuda.mem_get_info()
    if free < 2.5 * rows * 128 * 2:
        pytest.skip("needs 26 GB free")
    byte = torch.zeros((2, rows * 128), dtype=torch.uint8, device="cuda")
    scale = torch.zeros((2, rows // 64), device="cuda")
    view = lambda t, *s: t.view(torch.float8_e4m3fn).view(*s) if t.dtype == torch.uint8 else t.view(*s)  # noqa: E731
    flat = ad.KV8Cache(view(byte[0], 2, 1, L, 128), view(byte[1], 2, 1, L, 128), scale[0].view(2, 1, -1),
                       scale[1].view(2, 1, -1), 64)
    ws = ad.kv8_sparse_attention_workspace(2, 4, 1, 64)
    x = torch.randn((2, 2, 1, 128, 128), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    start = L - 128
    ad.kv8_append(flat, x[0], x[1], start, ws)
    k, v = ad.kv8_read(flat, start, 128, ws, torch.float32)
    q = _q(2, 4, torch.bfloat16, 5)
    idx = (start + torch.arange(64, device="cuda", dtype=torch.int32) * 2).expand(2, 4, 64).contiguous()
    out = ad.kv8_sparse_attention(q, flat, idx, ws)
    fine(ws)
    K, V = (t.double().cpu().numpy() for t in (k, v))
    C = scale[1].view(2, 1, -1)[:, :, start // 64:].double().cpu().numpy().repeat(64, 2)
    want, tol, _, _ = attention_oracle(q.double().cpu().numpy(), (K, V, C), lambda b, h: np.arange(64) * 2)
    check(out, want, tol, "sparse")
    for b in range(2):
        st, sc = ref.append(np.zeros((128, 128)), np.zeros(2), x[0, b, 0].double().cpu().numpy(), 0, "e4m3", 64)
        assert np.array_equal(K[b, 0], st * sc.repeat(64)[:, None])
    # the same memory as pages of 64 rows: a sequence on the last two pages
    pages = rows // 64
    paged = ad.KV8Cache(view(byte[0], pages, 1, 64, 128), view(byte[1], pages, 1, 64, 128),
                        scale[0].view(pages, 1, 1), scale[1].view(pages, 1, 1), 64,
                        block_table=i32([[pages - 2, pages - 1]]))
    dws = ad.kv8_attention_workspace(1, 4, 1, 128)
    out = ad.kv8_attention(q[1:], paged, i32([100]), dws)
    fine(dws)
    want, tol, _, _ = attention_oracle(q[1:].double().cpu().numpy(), (K[1:], V[1:], C[1:]),
                                       lambda b, h: np.arange(100))
    check(out, want, tol, "paged")
    # eviction in place moves the last page's rows down to the one before
    w = torch.zeros((1, 1, 128), device="cuda")
    w[..., 64:] = 1.0
    keep, lens = ad.kv8_evict(paged, w, i32([128]), 64, dws)
    fine(dws)
    assert keep[0, 0].tolist() == list(range(64, 128)) and lens.tolist() == [64]
    got, _ = ad.kv8_read(paged, 0, 64, dws, torch.float32)
    assert np.array_equal(got[0, 0].double().cpu().numpy(), K[1, 0, 64:])


def test_a_serving_step_in_one_graph():
    """append, sparse attention with weights and eviction into a second cache, captured together and
    replayed with new rows, queries and lengths: equal to eager calls."""
    B, Hkv, Hq, L, kk = 2, 2, 4, 256, 20
    base = Case(B, Hkv, L, "e4m3", block=16, seed=31)

    def setup():
        c = base.upload(ad)
        d = Case(B, Hkv, 96, "e4m3", block=16, empty=True).upload(ad)
        return dict(c=c, d=d, x=torch.zeros((2, B, Hkv, 1, D), dtype=torch.bfloat16, device="cuda"),
                    q=_q(B, Hq, torch.bfloat16), lens=i32([0, 0]), idx=i32([[[0] * kk] * Hq] * B),
                    w=torch.zeros((B, Hkv, L), device="cuda"), w2=torch.zeros((B, Hkv, 96), device="cuda"),
                    out=torch.empty((B, Hq, D), device="cuda"), lens2=i32([0, 0]), now=i32([0, 0]),
                    keep=torch.empty((B, Hkv, 90), dtype=torch.int32, device="cuda"),
                    ws=ad.kv8_sparse_attention_workspace(B, Hq, Hkv, kk, weights=True))

    def step(s):
        ad.PreparedKV8Append(s["c"], s["x"][0], s["x"][1], s["lens"], s["ws"])()
        torch.add(s["lens"], 1, out=s["now"])
        ad.PreparedKV8SparseAttention(s["q"], s["c"], s["idx"], s["ws"], s["out"], weights=s["w"])()
        ad.PreparedKV8Evict(s["c"], s["d"], s["w"], s["w2"], s["now"], s["lens2"], s["keep"], 90, 2, 8,
                            s["ws"])()

    a, b = setup(), setup()
    step(a)
    torch.cuda.synchronize()
    a = setup()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        step(a)
    rng = np.random.default_rng(3)
    for lens in ([100, 80], [200, 17], [255, 90]):
        x = torch.from_numpy(rng.standard_normal((2, B, Hkv, 1, D))).to(torch.bfloat16)
        idx = np.stack([np.stack([np.sort(rng.choice(n, min(n, kk), replace=False)) for _ in range(Hq)])
                        if n >= kk else np.tile(np.r_[0:n, [-1] * (kk - n)], (Hq, 1)) for n in lens])
        for s in (a, b):
            s["x"].copy_(x)
            s["q"].copy_(_q(B, Hq, torch.bfloat16, lens[0]))
            s["lens"].copy_(i32(lens))
            s["idx"].copy_(up(idx.astype(np.int32)))
        graph.replay()
        step(b)
        torch.cuda.synchronize()
        for n in ("out", "w", "w2", "lens2", "keep"):
            assert torch.equal(a[n], b[n]), n
        for n in ("c", "d"):
            assert torch.equal(a[n].k.view(torch.uint8), b[n].k.view(torch.uint8))
            assert torch.equal(a[n].v_scale, b[n].v_scale)
    fine(a["ws"])
    fine(b["ws"])


def test_append_of_broadcast_rows():
    """Stride 0: one row's values given to every head."""
    c = Case(1, 4, 32, "int8", block=8, seed=2)
    cache = c.upload(ad)
    x = torch.randn((1, 1, 5, D), generator=torch.Generator().manual_seed(0)).cuda().expand(1, 4, 5, D)
    ws = ad.kv8_workspace()
    ad.kv8_append(cache, x, x, 9, ws)
    fine(ws)
    k, ks, _, _, _ = c.download(cache)
    for h in range(4):
        st, sc = ref.append(c.k[0, h], c.ks[0, h], x[0, 0].double().cpu().numpy(), 9, "int8", 8)
        assert np.array_equal(k[0, h], st) and np.array_equal(ks[0, h], sc)


def test_a_larger_workspace_serves_smaller_calls():
    c = Case(1, 2, 300, "e4m3", block=16, seed=2)
    cache, q = c.upload(ad), _q(1, 8, torch.bfloat16)
    big = ad.kv8_attention_workspace(4, 32, 8, 4096, weights=True)
    small = ad.kv8_attention_workspace(1, 8, 2, cache.Lmax)
    for _ in range(2):
        a = ad.kv8_attention(q, cache, i32([300]), big)
        w = torch.zeros((1, 2, cache.Lmax), device="cuda")
        b = ad.kv8_attention(q, cache, i32([300]), big, weights=w)
        assert torch.equal(a, b) and torch.equal(a, ad.kv8_attention(q, cache, i32([300]), small))
    with pytest.raises(ad.AdamasError):
        ad.kv8_attention(q, cache, i32([300]), small, weights=w)
    fine(big)
