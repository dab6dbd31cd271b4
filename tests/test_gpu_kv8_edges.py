"""8-bit caches on the GPU at the ends of their value ranges, with bad pages and at the largest sizes,
against the float64 oracle (oracle/kv8_ref.py)."""
import numpy as np
import pytest
import torch

import oracle
import token_level_sparse_fwht_b200 as ad
from kv8_helpers import D, Case, attention_oracle, check
from oracle import kv8_ref as ref

pytestmark = pytest.mark.gpu
FMTS = ["e4m3", "int8"]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# -------------------------------------------------------------- attention: value ranges
def _leading_zero_block(fmt, block, lead, target, scale, seed):
    """A cache of 64 positions whose first block has zero V rows (stored with the smallest scale, or with
    scale 0) and scores `lead` powers of two above all others; the other blocks' largest |V| is `target`
    times 1, 1/8, ...  Returns the case and a query [1, 2, 128]."""
    c = Case(1, 1, 64, fmt, block=block, seed=seed, spread=0)
    top = ref.FMAX[fmt]
    c.v[:, :, :block] = 0
    c.vs[...] = target / top * 2.0 ** (-3.0 * (np.arange(64 // block) % 4 - 1).clip(min=0))
    c.vs = c.vs.astype(np.float32).astype(np.float64)
    c.vs[..., 0] = scale
    # dimension 0 alone leads: q_0 k_0 a log2(e) / sqrt(128) = lead
    c.k[..., 0] = 0
    c.k[:, :, :block] = 0
    c.k[:, :, :block, 0] = 64
    q = np.random.default_rng(seed).standard_normal((1, 2, D)) * 0.05
    q[..., 0] = 16
    c.ks[..., 0] = np.float32(lead * np.sqrt(D) / (16 * 64 * np.log2(np.e)))
    return c, torch.from_numpy(q)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("block", [4, 16])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lead", [60, 100, 111, 114, 120, 126, 150, 200])
@pytest.mark.parametrize("form", ["dense", "sparse", "shared"])
def test_zero_values_that_lead_leave_the_others_finite_and_right(fmt, block, dtype, lead, form):
    """The zero block's p is 1 and its values add nothing; the others' p is about 2^-lead and their values
    are large, so the output is theirs alone.  2^-125 is added to the bounds: fp32 results below
    its smallest normal number (2^-126) have fewer bits."""
    for target in (300.0, 1000.0, 1e6):
        for scale in (2.0 ** -126, 0.0):
            c, q = _leading_zero_block(fmt, block, lead, target, scale, seed=lead)
            q = q.to(dtype)
            want, tol, ww, wtol = attention_oracle(q.double().numpy(), c, lambda b, h: np.arange(64))
            cache, w = c.upload(ad), torch.zeros((1, 1, 64), device="cuda")
            if form == "dense":
                ws = ad.kv8_attention_workspace(1, 2, 1, cache.Lmax, weights=True)
                out = ad.kv8_attention(q.cuda(), cache, i32([64]), ws, weights=w)
            else:
                n = 1 if form == "shared" else 2
                idx = np.random.default_rng(1).permuted(np.tile(np.arange(64), (1, n, 1)), axis=-1)
                ws = ad.kv8_sparse_attention_workspace(1, 2, 1, 64, shared=form == "shared", weights=True)
                out = ad.kv8_sparse_attention(q.cuda(), cache, i32(idx.tolist()), ws,
                                              shared=form == "shared", weights=w)
            ad.check_workspace(ws)
            check(out, want, tol + 2.0 ** -125, (target, scale))
            check(w, ww, wtol + 2.0 ** -125, "weights")
            if lead <= 111:
                assert (np.abs(want) > 2.0 ** -122).any()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("e", [-126, -120, -110])
@pytest.mark.parametrize("L,block", [(25, 1), (1000, 16), (40000, 64)])
def test_many_keys_of_very_small_values(fmt, e, L, block):
    """Equal scores over L keys and value scales of 2^e: outputs are normal fp32 numbers (4 2^e and more)
    although 1 / L of the smallest scale is none.  The bound is the helper's alone."""
    c = Case(1, 2, L, fmt, block=block, seed=L, spread=0)
    c.v[:] = np.abs(c.v) + ref.FMAX[fmt] / 4
    c.v[:] = np.minimum(ref.round8(c.v, fmt), ref.FMAX[fmt])
    c.vs[:] = 2.0 ** e
    q = torch.zeros((1, 8, D), dtype=torch.bfloat16)
    want, tol, _, _ = attention_oracle(q.double().numpy(), c, lambda b, h: np.arange(L))
    assert (want > 4 * 2.0 ** e).all()
    ws = ad.kv8_attention_workspace(1, 8, 2, c.cap)
    out = ad.kv8_attention(q.cuda(), c.upload(ad), i32([L]), ws)
    ad.check_workspace(ws)
    check(out, want, tol, "out")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block", [4, 16])
@pytest.mark.parametrize("r", [0, 8, 16, 20, 24, 28])
def test_small_blocks_show_where_large_ones_hold_zeros(fmt, dtype, block, r):
    """p c is held in two fp16 parts under one reference per head: to 2^-22 of itself or 2^-37 of the
    head's largest (w > 2^12 at least there, and the second part's half step is 2^-25).  Half of
    the blocks have 2^r times the scale of the others and zeros in the upper dimensions, where the others
    hold positive values; there the bound is 2^(r - 37) of the output and what the sums drop."""
    L = 256
    c = Case(1, 1, L, fmt, block=block, seed=r, spread=0)
    c.ks[:] = 2.0 ** -6
    large = np.arange(L) // block % 2 == 0
    c.v[:, :, large, D // 2:] = 0
    c.v[:, :, ~large, D // 2:] = ref.round8(np.abs(c.v[:, :, ~large, D // 2:]) + 1, fmt)
    c.vs[:] = np.where(large[::block], 2.0 ** r, 1.0)
    q = torch.randn((1, 4, D), generator=torch.Generator().manual_seed(r)).to(dtype)
    want, tol, _, _ = attention_oracle(q.double().numpy(), c, lambda b, h: np.arange(L))
    # the bound (2^-9 of the largest p at r = 28, a few times the mean) is far under what is compared: a
    # block lost would show
    assert (tol[..., D // 2:] < 2.0 ** -6 * want[..., D // 2:]).all()
    cache = c.upload(ad)
    ws = ad.kv8_attention_workspace(1, 4, 1, L)
    out = ad.kv8_attention(q.cuda(), cache, i32([L]), ws)
    check(out, want, tol, "dense")
    sws = ad.kv8_sparse_attention_workspace(1, 4, 1, L)
    idx = np.random.default_rng(r).permuted(np.tile(np.arange(L), (1, 4, 1)), axis=-1)
    check(ad.kv8_sparse_attention(q.cuda(), cache, i32(idx.tolist()), sws), want, tol, "sparse")
    ad.check_workspace(ws)
    ad.check_workspace(sws)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("r", [0, 8, 14, 18])
def test_small_query_elements_show_where_keys_hold_zeros(fmt, dtype, r):
    """One element of q is 2^r times the others and meets zeros: scores come from the others alone, which
    are held to 2^-22 of themselves (in the helper's bound) or 2^-39 of the largest, in
    every product: |dx| <= 2^-39 max|q| a sum|k| / sqrt(d), and an output's change e^(2 dx) of
    its terms."""
    L = 200
    c = Case(1, 1, L, fmt, block=8, seed=r, spread=0)
    c.k[..., 3] = 0
    c.ks[:] = 2.0 ** -5
    q = torch.randn((1, 4, D), generator=torch.Generator().manual_seed(r))
    q[..., 3] = 2.0 ** r * 4
    q = q.to(dtype)
    want, tol, ww, wtol = attention_oracle(q.double().numpy(), c, lambda b, h: np.arange(L))
    K, V = c.values()
    dx = 2.0 ** -39 * q.abs().double().max().item() * np.abs(K[0, 0, :L]).sum(-1).max() / np.sqrt(D)
    assert dx < 2.0 ** -10
    tol = tol + 2.1 * dx * np.abs(V[0, 0, :L]).max(0)
    ws, w = ad.kv8_attention_workspace(1, 4, 1, c.cap, weights=True), torch.zeros((1, 1, c.cap), device="cuda")
    out = ad.kv8_attention(q.cuda(), c.upload(ad), i32([L]), ws, weights=w)
    ad.check_workspace(ws)
    check(out, want, tol, "out")
    check(w, ww, wtol + 2.1 * dx * ww + 2.0 ** -140, "weights")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block", [8, 32])
@pytest.mark.parametrize("e", [0, 10, 14, 16, 18, 20, 24, 40, 90])
@pytest.mark.parametrize("G", [2, 5])
def test_scores_of_any_size_choose_the_leading_keys(fmt, dtype, block, e, G):
    """Scores of about 2^10 2^e.  Every head has three keys that lead all others by more than the scores'
    rounding (20 units of 2^-23 of sum |q k|, and 40 for the exponential): copies of the head's
    query, one of them stored with half its bytes' size under twice the scale, so all products are
    equal.  The output is the mean of their three values, to the exponential's and the sums' last bits."""
    L = 700
    c = Case(1, 1, L, fmt, block=block, seed=e, spread=0)
    q = torch.randn((1, G, D), generator=torch.Generator().manual_seed(e)).to(dtype)
    c.ks[:] = 2.0 ** e
    lead = np.random.default_rng(e).permutation(c.cap // block - 2)[:3 * G].reshape(G, 3) * block + 1
    for h in range(G):
        x = q[0, h].double().numpy()
        row = ref.round8(x / np.abs(x).max() * ref.FMAX[fmt] / 4, fmt) * 2
        for n, p in enumerate(lead[h]):
            c.k[0, 0, p] = row / 2 if n == 1 else row
            if n == 1:
                c.ks[0, 0, p // block] = 2.0 ** (e + 1)
                c.k[0, 0, p + 1:p // block * block + block] /= 2
                c.k[0, 0, p // block * block:p] /= 2
                c.k[0, 0, p // block * block:][:block] = ref.round8(c.k[0, 0, p // block * block:][:block], fmt)
    K, V = (x[0, 0, :L] for x in c.values())
    want, others, S = np.zeros((1, G, D)), np.ones((G, L), bool), 0.0
    for h in range(G):
        x = K @ q[0, h].double().numpy() / np.sqrt(D)
        others[h, lead[h]] = False
        S = (np.abs(K) @ np.abs(q[0, h].double().numpy())).max() / np.sqrt(D)
        assert np.ptp(x[lead[h]]) == 0 and x[lead[h][0]] - x[others[h]].max() > 20 * 2.0 ** -23 * S + 40
        want[0, h] = V[lead[h]].mean(0)
    tol = np.broadcast_to(2.0 ** -20 * np.abs(V).max(), want.shape)
    cache, lens = c.upload(ad), i32([L])
    ws = ad.kv8_attention_workspace(1, G, 1, c.cap, weights=True)
    w = torch.zeros((1, 1, c.cap), device="cuda")
    check(ad.kv8_attention(q.cuda(), cache, lens, ws, weights=w), want, tol, "dense")
    ww = np.zeros((1, 1, c.cap))
    np.add.at(ww[0, 0], lead.ravel(), 1 / 3)
    check(w, ww, np.full_like(ww, 2.0 ** -20), "weights")
    sws, w = ad.kv8_sparse_attention_workspace(1, G, 1, L, weights=True), torch.zeros_like(w)
    idx = np.random.default_rng(1).permuted(np.tile(np.arange(L), (1, G, 1)), axis=-1)
    check(ad.kv8_sparse_attention(q.cuda(), cache, i32(idx.tolist()), sws, weights=w), want, tol, "sparse")
    check(w, ww, np.full_like(ww, 2.0 ** -20), "sparse weights")
    ad.check_workspace(ws)
    ad.check_workspace(sws)


# ----------------------------------------------------------------- eviction: bad pages
# Positions 32 .. 47 of sequence 0 are on a page that does not exist.  Kept lists whose rows from there
# are the first of a block, in its middle and its end, several blocks, and a whole block.
GAPS = [[*range(8), 40, *range(48, 63)],
        [*range(7), *range(33, 42), *range(48, 56)],
        [3, 5, 36, 37, *range(50, 70)],
        [*range(32, 48), *range(60, 68)],
        [*range(0, 31, 2), 47]]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("block", [1, 4, 8, 16])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kept", GAPS)
def test_evict_leaves_out_only_the_rows_of_a_bad_page(fmt, block, in_place, kept):
    c = Case(2, 2, 96, fmt, block=block, page=16, seed=7, codes=True, spread=6)
    c.codes[:] = np.random.default_rng(3).integers(0, 256, c.codes.shape, dtype=np.uint8)
    cache = c.upload(ad)
    cache.block_table[0, 2] = c.num_pages + 3
    n = len(kept)
    d, kw = c, {}
    if not in_place:
        d = Case(2, 2, n, fmt, block=block, page=16, seed=8, codes=True)
        kw = dict(dst=d.upload(ad))
    w = torch.zeros((2, 2, cache.Lmax), device="cuda")
    w[..., kept] = 1.0
    before, ws = d.download(kw.get("dst", cache)), ad.kv8_workspace()
    keep, lens = ad.kv8_evict(cache, w, i32([96, 96]), n, ws, **kw)
    with pytest.raises(ad.AdamasError) as err:
        ad.check_workspace(ws)
    assert err.value.status == ad.ERR_INVALID_ARG
    assert (keep.cpu() == torch.tensor(kept)).all() and lens.tolist() == [n, n]
    got, vals = d.download(kw.get("dst", cache)), c.values()
    for b in range(2):
        came = np.array([b == 1 or not 32 <= p < 48 for p in kept])
        for h in range(2):
            for i in (0, 2):
                for r in range(0, n, block):
                    rows, ok = slice(r, min(r + block, n)), came[r:min(r + block, n)]
                    was, now = before[i][b, h, rows], got[i][b, h, rows]
                    assert np.array_equal(now[~ok], was[~ok]), (b, h, i, r)
                    s = got[i + 1][b, h, r // block]
                    if not ok.any():
                        assert s == before[i + 1][b, h, r // block]
                        continue
                    stored, scale = ref.requantise(vals[i // 2][b, h, np.array(kept)[rows][ok]], fmt, block)
                    assert np.array_equal(now[ok] * s, stored * scale[0]), (b, h, i, r)
            want = c.codes[b, h, kept]
            want[~came] = before[4][b, h, :n][~came]
            assert np.array_equal(got[4][b, h, :n], want)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block", [4, 16])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_keeps_values_at_fp32s_largest(fmt, dtype, block, in_place):
    """Appended values next to the type's largest are rounded up to 2^128, which the bytes and the scale hold and
    fp32 does not; the move keeps them, and what shares their block."""
    L = 64
    x = np.random.default_rng(block).standard_normal((1, 2, L, D)) * 2.0 ** 118
    x = torch.from_numpy(x).to(dtype)
    x[:, :, ::3, 5] = torch.finfo(dtype).max
    x[:, 1, ::7, 9] = -torch.finfo(dtype).max
    c = Case(1, 2, L, fmt, block=block, empty=True)
    cache, ws = c.upload(ad), ad.kv8_workspace()
    ad.kv8_append(cache, x.cuda(), x.cuda(), 0, ws)
    k, ks, v, vs, _ = c.download(cache)
    for h in range(2):
        want, sc = ref.append(np.zeros((L, D)), np.zeros(L // block), x[0, h].double().numpy(), 0, fmt, block)
        assert np.array_equal(k[0, h], want) and np.array_equal(ks[0, h], sc)
    kept = [*range(3, 20), *range(30, 63, 2)]
    w = torch.zeros((1, 2, L), device="cuda")
    w[..., kept] = 1.0
    n = len(kept)
    d = c if in_place else Case(1, 2, n, fmt, block=block, empty=True)
    kw = {} if in_place else dict(dst=d.upload(ad))
    ad.kv8_evict(cache, w, i32([L]), n, ws, **kw)
    ad.check_workspace(ws)
    got = d.download(kw.get("dst", cache))
    for i, (st, sc) in ((0, (k, ks)), (2, (v, vs))):
        for h in range(2):
            vals = (st[0, h] * sc[0, h].repeat(block)[:, None])[kept]
            assert np.abs(vals).max() == 2.0 ** 128
            want, scale = ref.requantise(vals, fmt, block)
            have = got[i][0, h, :n] * got[i + 1][0, h].repeat(block)[:n, None]
            assert np.array_equal(have, want * scale.repeat(block)[:n, None]), (i, h)


# --------------------------------------------------------------------------- binding
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float64])
def test_calls_do_not_depend_on_torchs_default_type(dtype):
    """A model's program often sets its own default type; what the calls make is float32 where it has to be."""
    rng = np.random.default_rng(4)
    x = torch.from_numpy(rng.standard_normal((2, 1, 2, 96, D))).to(torch.bfloat16).cuda()
    q, w = torch.from_numpy(rng.standard_normal((1, 4, D))).float().cuda(), torch.rand((1, 2, 96), device="cuda")
    idx = i32(rng.permuted(np.tile(np.arange(96), (1, 4, 1)), axis=-1)[..., :40].tolist())

    def run():
        cache, dst = (ad.kv8_cache(1, 2, n, block_size=16) for n in (96, 48))
        ws = ad.kv8_attention_workspace(1, 4, 2, 96, weights=True)
        ad.kv8_append(cache, x[0], x[1], 0, ws)
        sums = w.clone()
        outs = [ad.kv8_attention(q, cache, None, ws, weights=sums),
                ad.kv8_sparse_attention(q, cache, idx, ad.kv8_sparse_attention_workspace(1, 4, 2, 40))]
        keep, lens = ad.kv8_evict(cache, sums, i32([96]), 48, ws, sink=1, recent=5, dst=dst)
        outs += [sums, keep, lens, *ad.kv8_read(dst, 0, 48, ws)]
        ad.check_workspace(ws)
        return outs

    want, was = run(), torch.get_default_dtype()
    torch.set_default_dtype(dtype)
    try:
        got = run()
    finally:
        torch.set_default_dtype(was)
    assert all(torch.equal(a, b) and a.dtype == b.dtype for a, b in zip(got, want))


@pytest.mark.parametrize("B,Hkv,n", [(2, 4, 1), (1, 4, 3), (3, 1, 5), (1, 1, 1)])
def test_append_ignores_the_strides_of_dimensions_of_one_element(B, Hkv, n):
    """One token a step: K a head-major tensor, V a slice of a token-major one, rows alike."""
    rng = np.random.default_rng(B)
    k = torch.from_numpy(rng.standard_normal((B, Hkv, n, D))).to(torch.bfloat16).cuda()
    v = torch.empty((B, n, Hkv, D), dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    if B == 1:                                        # one row of a batch laid out otherwise
        v = torch.empty((2, Hkv, n, D), dtype=torch.bfloat16, device="cuda")[:1].as_strided(
            (1, Hkv, n, D), (7, n * D, D, 1))
    if Hkv == 1:
        v = torch.empty((B, n, D), dtype=torch.bfloat16, device="cuda").as_strided(
            (B, 1, n, D), (n * D, 24, D, 1))
    v.copy_(-k)
    a, b = (ad.kv8_cache(B, Hkv, 32, block_size=8, dtype=torch.int8) for _ in range(2))
    ws = ad.kv8_workspace()
    ad.kv8_append(a, k, v, 9, ws)
    ad.kv8_append(b, k, (-k).contiguous(), 9, ws)
    ad.check_workspace(ws)
    for x, y in ((a.k, b.k), (a.v, b.v), (a.k_scale, b.k_scale), (a.v_scale, b.v_scale)):
        assert torch.equal(x, y)
    assert torch.equal(a.v, -a.k)


@pytest.mark.parametrize("dtype,wide,first", [(torch.bfloat16, 132, 0), (torch.bfloat16, 136, 4),
                                              (torch.float32, 130, 0), (torch.float32, 132, 2)])
def test_append_names_rows_that_do_not_start_at_16_bytes(dtype, wide, first):
    x = torch.zeros((1, 2, 3, wide), dtype=dtype, device="cuda")[..., first:first + D]
    with pytest.raises(ValueError, match="16 bytes"):
        ad.kv8_append(ad.kv8_cache(1, 2, 32, block_size=8), x, x, 0, ad.kv8_workspace())


# ------------------------------------------------------------------- the longest selections
@pytest.mark.parametrize("B,L,budget,sink,recent", [(1, 393216, 1000, 0, 0), (1, 393217, 200000, 7, 1000),
                                                    (2, 600001, 50001, 0, 64), (1, 786432, 300000, 4, 5000),
                                                    (1, 786432, 786431, 0, 0), (1, 786432, 17, 3, 14)])
def test_evict_select_of_the_longest_sequences(B, L, budget, sink, recent):
    """Clusters of 8 and of 16 CTAs; a tie over about a third of the positions crosses every share."""
    rng = np.random.default_rng(budget)
    w = rng.random((B, 1, L)).astype(np.float32)
    w[rng.random((B, 1, L)) < 1 / 3] = 0.75
    w[..., rng.integers(0, L, 50)] = np.nan
    lens = [L, L - 77777][:B]
    ws, out = ad.kv8_workspace(), torch.from_numpy(w).cuda()
    keep = ad.evict_select(out, i32(lens), budget, ws, sink=sink, recent=recent, weights_out=out)
    ad.check_workspace(ws)
    keep, out = keep.cpu().numpy(), out.cpu().numpy()
    for b in range(B):
        want = ref.evict_select(w[b, 0], lens[b], budget, sink, recent)
        n = len(want)
        assert np.array_equal(keep[b, 0, :n], want) and (keep[b, 0, n:] == -1).all()
        assert np.array_equal(out[b, 0, :n], w[b, 0, want], equal_nan=True)
        assert (out[b, 0, n:lens[b]] == 0).all()
        assert np.array_equal(out[b, 0, lens[b]:], w[b, 0, lens[b]:], equal_nan=True)


def test_evict_of_a_long_cache():
    """Selection by 16 CTAs, then the move in place, against the definition."""
    L, budget = 400000, 9000
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = ad.kv8_cache(1, 1, L, block_size=64)
    x = torch.randn((1, 1, L, D), generator=g, device="cuda", dtype=torch.float32)
    ws = ad.kv8_workspace()
    ad.kv8_append(cache, x, -x, 0, ws)
    k, v = ad.kv8_read(cache, 0, L, ws, dtype=torch.float32)
    w = torch.rand((1, 1, cache.Lmax), generator=g, device="cuda")
    want = ref.evict_select(w[0, 0].cpu().numpy(), L, budget, 4, 256)
    keep, lens = ad.kv8_evict(cache, w, i32([L]), budget, ws, sink=4, recent=256)
    ad.check_workspace(ws)
    assert np.array_equal(keep[0, 0].cpu().numpy(), want) and lens.tolist() == [budget]
    for got, old in zip(ad.kv8_read(cache, 0, budget, ws, dtype=torch.float32), (k, v)):
        stored, scale = ref.requantise(old[0, 0, keep[0, 0].long()].double().cpu().numpy(), "e4m3", 64)
        assert np.array_equal(got[0, 0].double().cpu().numpy(), stored * scale.repeat(64)[:budget, None])


# ------------------------------------------------------------------------- codes of append
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("block", [1, 8, 16, 64, 256])
@pytest.mark.parametrize("kw", [dict(t=1.01), dict(ratio=0.5)])
def test_append_codes_of_every_form(dtype, fmt, block, kw):
    """Rows from inside a block on, over several blocks: the codes are the definition's and the encoder's but
    for coordinates next to a threshold (fp32 sums of 128: within 1e-4 of the vector's scale, as for
    the encoder), other positions keep theirs."""
    B, Hkv, L, n = 2, 2, 512, 300
    starts, counts = [5, 201], [n, 77]
    c = Case(B, Hkv, L, fmt, block=block, seed=block, codes=True)
    c.codes[:] = np.random.default_rng(1).integers(0, 256, c.codes.shape, dtype=np.uint8)
    x = torch.from_numpy(np.random.default_rng(block + 1).standard_normal((B, Hkv, n, D)) * 1.3).to(dtype)
    x[:, :, ::5] *= 8
    cache, ws = c.upload(ad), ad.kv8_workspace()
    ad.kv8_append(cache, x.cuda(), x.cuda(), i32(starts), ws, counts=i32(counts), **kw)
    ad.check_workspace(ws)
    codes = c.download(cache)[4]
    enc = torch.zeros((B, Hkv, n, 32), dtype=torch.uint8, device="cuda")
    if "t" in kw:
        ad.encode_keys(x.cuda(), enc, 0, n, kw["t"])
    else:
        ad.encode_keys_absmax(x.cuda(), enc, 0, n, kw["ratio"])
    for b in range(B):
        rows = x[b, :, :counts[b]].double().numpy()
        y = oracle.hadamard_rotate(rows)
        if "t" in kw:
            want, margin = oracle.bucketize(y, kw["t"]), oracle.threshold_margin(y, kw["t"])
        else:
            t = oracle.absmax_thresholds(rows, kw["ratio"])
            want = oracle.bucketize_per_vector(y, t)
            margin = np.minimum(np.abs(np.abs(y) - np.asarray(t).reshape(*y.shape[:-1], 1)), np.abs(y))
        near = margin < 1e-4 * np.maximum(1.0, np.abs(y).max(-1, keepdims=True))
        got = oracle.unpack_codes(codes[b, :, starts[b]:starts[b] + counts[b]])
        theirs = oracle.unpack_codes(enc[b, :, :counts[b]].cpu().numpy())
        assert not ((got != want) & ~near).any() and not ((got != theirs) & ~near).any()
        rest = np.ones(c.cap, bool)
        rest[starts[b]:starts[b] + counts[b]] = False
        assert np.array_equal(codes[b][:, rest], c.codes[b][:, rest])


def test_evict_of_more_sums_than_32_bits_count():
    """1024 sequences x 16 kv heads x 131072 positions are 2^31 running sums, although the sequences here
    are short and hold a page each: the cache's own rows are few."""
    B, H, page, L, budget = 1024, 16, 64, 131072, 24
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randint(0, 256, (B, H, page, D), generator=g, device="cuda", dtype=torch.uint8)
            .view(torch.int8).clamp(-127, 127) for _ in range(2))
    ks, vs = (torch.exp2(torch.randint(-6, 6, (B, H, page // 16), generator=g, device="cuda").float())
              for _ in range(2))
    table = torch.randperm(B, generator=g, device="cuda").int()[:, None].expand(-1, L // page).contiguous()
    cache, ws = ad.KV8Cache(k, v, ks, vs, 16, block_table=table), ad.kv8_workspace()
    assert cache.Lmax == L
    old = ad.kv8_read(cache, 0, page, ws, dtype=torch.float32)
    w = torch.zeros((B, H, L), device="cuda")
    sums = torch.rand((B, H, page), generator=g, device="cuda")
    w[..., :page] = sums
    lens = torch.randint(0, page + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    lens[-1] = page
    was = lens.tolist()
    keep, _ = ad.kv8_evict(cache, w, lens, budget, ws, sink=2, recent=5)
    ad.check_workspace(ws)
    new = ad.kv8_read(cache, 0, budget, ws, dtype=torch.float32)
    for b in (0, 1, 511, 700, B - 1):
        for h in (0, H - 1):
            want = ref.evict_select(sums[b, h].cpu().numpy(), was[b], budget, 2, 5)
            n = len(want)
            assert np.array_equal(keep[b, h, :n].cpu().numpy(), want) and lens[b].item() == n
            assert torch.equal(w[b, h, :n], sums[b, h, want]) and not w[b, h, n:was[b]].any()
            assert torch.equal(w[b, h, was[b]:page], sums[b, h, was[b]:])   # behind a sequence: left
            for x, y in zip(new, old):
                stored, scale = ref.requantise(y[b, h, want].double().cpu().numpy(), "int8", 16)
                if was[b] > budget:
                    assert np.array_equal(x[b, h, :n].double().cpu().numpy(), stored * scale.repeat(16)[:n, None])
                else:
                    assert torch.equal(x[b, h, :n], y[b, h, :n])
