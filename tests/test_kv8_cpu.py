"""8-bit caches without a GPU: the oracle against other means, the entry points' refusals (all on
the host, before any launch) and the binding's checks."""
import ctypes
import math

import numpy as np
import pytest
import torch

import token_level_sparse_fwht_b200 as ad
from kv8_helpers import Case, quantise, to_bytes
from oracle import kv8_ref as ref
from token_level_sparse_fwht_b200 import BF16, ERR_INVALID_ARG, ERR_UNSUPPORTED
from token_level_sparse_fwht_b200.kv8 import _CCache, _new_workspace

A = 1 << 20          # a fake, 256-byte aligned "device" address; never dereferenced


# ------------------------------------------------------------------------- oracle
def test_e4m3_values_are_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(ref.e4m3_values(), t.astype(np.float64), equal_nan=True)


def test_round8_is_the_nearest_value_ties_to_even():
    vals = ref.e4m3_values()
    pos = np.unique(np.abs(vals[np.isfinite(vals)]))
    mids = (pos[1:] + pos[:-1]) / 2
    x = np.concatenate([pos, mids, mids * (1 + 1e-9), mids * (1 - 1e-9),
                        np.random.default_rng(0).standard_normal(5000) * 50, [1e3, -1e9]])
    want = torch.from_numpy(np.clip(x, -448, 448).astype(np.float64)).to(torch.float32)
    keep = want.double().numpy() == np.clip(x, -448, 448)            # what float32 holds exactly
    got = ref.round8(x, "e4m3")
    assert np.array_equal(got[keep], want.to(torch.float8_e4m3fn).double().numpy()[keep])
    d = np.abs(np.clip(x, -448, 448)[:, None] - np.concatenate([pos, -pos])[None])
    assert np.allclose(np.abs(got - np.clip(x, -448, 448)), d.min(1), atol=0)
    assert ref.round8([0.5, 1.5, -2.5, 126.6, 300, -300], "int8").tolist() == [0, 2, -2, 127, 127, -127]


@pytest.mark.parametrize("fmt,top", [("e4m3", 448.0), ("int8", 127.0)])
def test_block_scale_borders(fmt, top):
    a = np.array([0.0, 1e-45, top, np.nextafter(top, 1e9), top * 2.0 ** -126, top * 2.0 ** 100, 1.0])
    s = ref.block_scale(a, fmt)
    assert s[0] == s[1] == 2.0 ** -126 and s[2] == 1 and s[3] == 2 and s[4] == 2.0 ** -126
    assert s[5] == 2.0 ** 100 and s[6] == (2.0 ** -8 if fmt == "e4m3" else 2.0 ** -6)
    assert (a <= top * s).all()


def test_attention_oracle_is_torchs_and_select_is_topk():
    rng = np.random.default_rng(1)
    q, K, V = rng.standard_normal(128), rng.standard_normal((50, 128)), rng.standard_normal((50, 128))
    want = torch.nn.functional.scaled_dot_product_attention(
        *(torch.from_numpy(x) for x in (q[None, None], K[None], V[None])))
    assert np.allclose(ref.attention(q, K, V, np.arange(50))[0], want[0, 0].numpy(), atol=1e-13)
    w = rng.standard_normal(200)
    got = ref.evict_select(w, 200, 60, 5, 20)
    mid = torch.from_numpy(w[5:180]).topk(35).indices.numpy() + 5
    assert np.array_equal(got, np.sort(np.concatenate([np.arange(5), mid, np.arange(180, 200)])))
    assert ref.evict_select(np.zeros(10), 10, 4, 0, 1).tolist() == [0, 1, 2, 9]


def test_append_in_pieces_within_a_blocks_scale_is_append_at_once():
    """With the largest row first no scale grows later: any cut gives the same cache."""
    rng = np.random.default_rng(2)
    x = rng.standard_normal((32, 128))
    x[::8] *= 4
    whole = ref.append(np.zeros((32, 128)), np.zeros(4), x, 0, "e4m3", 8)
    s = (np.zeros((32, 128)), np.zeros(4))
    for a, b in ((0, 3), (3, 4), (4, 19), (19, 32)):
        s = ref.append(*s, x[a:b], a, "e4m3", 8)
    assert np.array_equal(s[0], whole[0]) and np.array_equal(s[1], whole[1])
    st, sc = quantise(x, 8, "e4m3")
    assert np.array_equal(st, whole[0]) and np.array_equal(sc, whole[1])
    assert np.array_equal(to_bytes(st, "e4m3").double().numpy(), st)


# --------------------------------------------------------------------------- ABI
def cache(**kw):
    c = _CCache()
    d = dict(k=A, v=A + 4096, k_scale=A, v_scale=A, codes=None, block_table=None, Lmax=4096,
             num_pages=0, format=0, block_size=64, B=2, Hkv=8, d=128, page_size=0,
             max_blocks_per_seq=0, reserved=0)
    d.update(kw)
    for n, v in d.items():
        setattr(c, n, v)
    return ctypes.byref(c)


PAGED = dict(page_size=64, num_pages=100, block_table=A, max_blocks_per_seq=64)
BAD_CACHES = [
    (dict(k=None), ERR_INVALID_ARG), (dict(v=None), ERR_INVALID_ARG),
    (dict(k_scale=None), ERR_INVALID_ARG), (dict(v_scale=None), ERR_INVALID_ARG),
    (dict(k=A + 8), ERR_INVALID_ARG), (dict(v=A + 1), ERR_INVALID_ARG),
    (dict(k_scale=A + 2), ERR_INVALID_ARG), (dict(codes=A + 4), ERR_INVALID_ARG),
    (dict(format=2), ERR_INVALID_ARG), (dict(reserved=1), ERR_INVALID_ARG),
    (dict(block_size=0), ERR_INVALID_ARG), (dict(block_size=48), ERR_INVALID_ARG),
    (dict(block_size=512), ERR_INVALID_ARG), (dict(Lmax=4100), ERR_INVALID_ARG),
    (dict(Lmax=0), ERR_INVALID_ARG), (dict(B=0), ERR_INVALID_ARG), (dict(Hkv=-1), ERR_INVALID_ARG),
    (dict(d=64), ERR_UNSUPPORTED), (dict(Lmax=1 << 31), ERR_UNSUPPORTED),
    (dict(B=1 << 20, Hkv=32), ERR_UNSUPPORTED), (dict(block_table=A), ERR_INVALID_ARG),
    (dict(PAGED, page_size=48), ERR_INVALID_ARG), (dict(PAGED, page_size=32), ERR_INVALID_ARG),
    (dict(PAGED, page_size=-64), ERR_INVALID_ARG), (dict(PAGED, page_size=1 << 21), ERR_INVALID_ARG),
    (dict(PAGED, num_pages=0), ERR_INVALID_ARG), (dict(PAGED, block_table=None), ERR_INVALID_ARG),
    (dict(PAGED, block_table=A + 2), ERR_INVALID_ARG),
    (dict(PAGED, max_blocks_per_seq=63), ERR_INVALID_ARG),
]


def _append(c, **kw):
    a = dict(k=A, v=A, dt=BF16, n=16, sb=0, sh=128, sn=1024, starts=A, counts=None, t=1.0, ratio=0.0,
             ws=A, wb=256, stream=None)
    a.update(kw)
    return ad.lib().adamas_kv8_append(c, *a.values())


def _read(c, **kw):
    a = dict(starts=A, n=16, dt=BF16, k=A, v=A, ws=A, wb=256, stream=None)
    a.update(kw)
    return ad.lib().adamas_kv8_read(c, *a.values())


def _dense(c, **kw):
    a = dict(q=A, dt=BF16, c=c, Hq=32, lens=A, ws=A, wb=1 << 30, w_in=None, w_out=None, out=A, stream=None)
    a.update(kw)
    return ad.lib().adamas_kv8_attention(*a.values())


def _sparse(c, **kw):
    a = dict(q=A, dt=BF16, c=c, Hq=32, idx=A, k=128, shared=0, ws=A, wb=1 << 30, w_in=None, w_out=None,
             out=A, stream=None)
    a.update(kw)
    return ad.lib().adamas_kv8_sparse_attention(*a.values())


def _evict(c, **kw):
    a = dict(src=c, dst=c, w_in=A, w_out=A, lens=A, lens_out=A, budget=1000, sink=4, recent=100, keep=A,
             ws=A, wb=256, stream=None)
    a.update(kw)
    return ad.lib().adamas_kv8_evict(*a.values())


@pytest.mark.parametrize("call", [_append, _read, _dense, _sparse, _evict])
@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches_are_refused(call, kw, status):
    assert call(cache(**kw)) == status


@pytest.mark.parametrize("call", [_append, _read, _dense, _sparse, _evict])
def test_no_cache_is_refused(call):
    assert call(None) == ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(starts=None), dict(dt=2), dict(n=0),
                                dict(n=4097), dict(sn=4), dict(sh=-128), dict(sb=1 << 41), dict(k=A + 8),
                                dict(starts=A + 1), dict(counts=A + 2), dict(ws=None), dict(ws=A + 16),
                                dict(wb=255)])
def test_append_refusals(kw):
    assert _append(cache(), **kw) == ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(t=-1.0), dict(t=math.nan), dict(t=math.inf), dict(ratio=1.5),
                                dict(ratio=-0.5), dict(ratio=math.nan)])
def test_append_threshold_refusals(kw):
    assert _append(cache(codes=A), **kw) == ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(starts=None), dict(k=None), dict(v=None), dict(n=0), dict(dt=9),
                                dict(k=A + 4), dict(starts=A + 2), dict(ws=None), dict(wb=0)])
def test_read_refusals(kw):
    assert _read(cache(), **kw) == ERR_INVALID_ARG


ATT = [(dict(q=None), ERR_INVALID_ARG), (dict(out=None), ERR_INVALID_ARG), (dict(dt=3), ERR_INVALID_ARG),
       (dict(Hq=0), ERR_INVALID_ARG), (dict(Hq=33), ERR_INVALID_ARG), (dict(Hq=72), ERR_UNSUPPORTED),
       (dict(q=A + 8), ERR_INVALID_ARG), (dict(out=A + 8), ERR_INVALID_ARG), (dict(ws=None), ERR_INVALID_ARG),
       (dict(ws=A + 64), ERR_INVALID_ARG), (dict(wb=256), ERR_INVALID_ARG),
       (dict(w_in=A), ERR_INVALID_ARG), (dict(w_out=A), ERR_INVALID_ARG),
       (dict(w_in=A, w_out=A + 1), ERR_INVALID_ARG)]


@pytest.mark.parametrize("kw,status", ATT + [(dict(lens=A + 2), ERR_INVALID_ARG)])
def test_dense_refusals(kw, status):
    assert _dense(cache(), **kw) == status


@pytest.mark.parametrize("kw,status", ATT + [(dict(idx=None), ERR_INVALID_ARG), (dict(k=0), ERR_INVALID_ARG),
                                             (dict(shared=2), ERR_INVALID_ARG),
                                             (dict(idx=A + 2), ERR_INVALID_ARG)])
def test_sparse_refusals(kw, status):
    assert _sparse(cache(), **kw) == status


def test_attention_needs_the_workspace_its_size_function_names():
    for w in (0, 1):
        n = ad.lib().adamas_kv8_attention_workspace_bytes(2, 32, 8, 128, 4096, w)
        assert n > 0 and n % 256 == 0
        kw = dict(w_in=A, w_out=A) if w else {}
        assert _dense(cache(), wb=n - 1, **kw) == ERR_INVALID_ARG
    small = ad.lib().adamas_kv8_attention_workspace_bytes(2, 32, 8, 128, 4096, 0)
    assert _dense(cache(), wb=small, w_in=A, w_out=A) == ERR_INVALID_ARG
    f = ad.lib().adamas_kv8_attention_workspace_bytes
    for bad in ((0, 32, 8, 128, 64, 0), (1, 31, 8, 128, 64, 0), (1, 72, 8, 128, 64, 0), (1, 32, 8, 64, 64, 0),
                (1, 32, 8, 128, 0, 0), (1, 32, 8, 128, 64, 2), (1, 32, 8, 128, 1 << 31, 0)):
        assert f(*bad) == 0, bad
    g = ad.lib().adamas_kv8_sparse_attention_workspace_bytes
    assert g(1, 32, 8, 128, 128, 0, 0) > 0 and g(1, 32, 8, 128, 128, 1, 1) > g(1, 32, 8, 128, 128, 1, 0)
    assert g(1, 32, 8, 128, 0, 0, 0) == 0 and g(1, 32, 8, 128, 128, 2, 0) == 0
    with pytest.raises(ad.AdamasError):
        _new_workspace(0, "x", "cpu", None)


def test_evict_refusals():
    other = dict(k=A + (1 << 24), v=A + (1 << 25), k_scale=A + (1 << 26), v_scale=A + (1 << 27))
    assert _evict(cache(), dst=None) == ERR_INVALID_ARG
    for kw in (dict(w_in=None), dict(w_out=None), dict(lens=None), dict(lens_out=None), dict(keep=None),
               dict(budget=0), dict(sink=-1), dict(recent=-1), dict(sink=901), dict(budget=4097),
               dict(keep=A + 1), dict(lens_out=A + 1), dict(ws=None), dict(wb=128)):
        assert _evict(cache(), **kw) == ERR_INVALID_ARG, kw
    for kw in (dict(format=1), dict(B=1), dict(Hkv=4), dict(Lmax=960), dict(codes=A)):
        assert _evict(cache(), dst=cache(**other, **kw)) == ERR_INVALID_ARG, kw
    # some buffers shared, others not; or in place with another layout
    for kw in (dict(other, k=A), dict(other, v=A + 4096), dict(block_size=32), dict(Lmax=2048)):
        assert _evict(cache(), dst=cache(**kw)) == ERR_INVALID_ARG, kw
    assert _evict(cache(codes=A), dst=cache(**other, codes=A)) == ERR_INVALID_ARG
    long = dict(Lmax=1 << 20)
    assert _evict(cache(**long), dst=cache(**long)) == ERR_UNSUPPORTED


def test_evict_select_and_compact_refusals():
    f = ad.lib().adamas_evict_select
    ok = [A, 2, 8, 4096, A, 1000, 4, 100, A, None, 0, A, 256, None]
    for i, bad in [(0, None), (0, A + 2), (1, 0), (2, 0), (3, 0), (4, None), (4, A + 1), (5, 0), (5, 103),
                   (6, -1), (7, -1), (8, None), (8, A + 3), (11, None), (11, A + 8), (12, 255)]:
        a = list(ok); a[i] = bad
        assert f(*a) == ERR_INVALID_ARG, (i, bad)
    for out, top in ((A + (1 << 24), 999), (A, 2048), (A + 2, 4096)):
        a = list(ok); a[9], a[10] = out, top
        assert f(*a) == ERR_INVALID_ARG, (out, top)
    a = list(ok); a[3] = 786433
    assert f(*a) == ERR_UNSUPPORTED
    g = ad.lib().adamas_compact_rows
    ok = [A, A, 256, 2, 8, 4096, 0, 0, None, 0, A, 1000, A, A, 256, None]
    for i, bad in [(0, None), (1, None), (0, A + 8), (2, 64), (3, 0), (5, 0), (6, 48), (6, 16), (8, A),
                   (10, None), (10, A + 2), (11, 0), (11, 4097), (12, None), (13, None), (14, 0)]:
        a = list(ok); a[i] = bad
        assert g(*a) == ERR_INVALID_ARG, (i, bad)


def test_buffers_that_overlap_in_part_are_refused():
    far = dict(k=A + (1 << 24), v=A + (1 << 25), k_scale=A + (1 << 26), v_scale=A + (1 << 27))
    rows = 2 * 8 * 4096
    for kw in (dict(k=A + 128 * (rows - 1)), dict(v=A + 4096), dict(k_scale=A + 256), dict(v_scale=A + 128 * rows - 4)):
        assert _evict(cache(), dst=cache(**{**far, **kw})) == ERR_INVALID_ARG, kw
    n = 2 * 8 * 4096 * 4
    assert _evict(cache(), dst=cache(), w_in=A, w_out=A + n - 4) == ERR_INVALID_ARG
    for att in (_dense, _sparse):
        assert att(cache(), w_in=A, w_out=A + n - 4, wb=1 << 40) == ERR_INVALID_ARG
    f = ad.lib().adamas_evict_select
    assert f(A, 2, 8, 4096, A, 1000, 4, 100, A, A + 4096, 2048, A, 256, None) == ERR_INVALID_ARG
    g = ad.lib().adamas_compact_rows
    assert g(A, A + 256 * (rows - 1), 256, 2, 8, 4096, 0, 0, None, 0, A, 1000, A, A, 256, None) == ERR_INVALID_ARG
    # paged: as many rows as there are pages
    assert g(A, A + 256 * 31, 256, 2, 1, 32, 16, 2, A, 2, A, 10, A, A, 256, None) == ERR_INVALID_ARG


# ----------------------------------------------------------------------- binding
def test_binding_refuses_host_tensors_and_wrong_shapes():
    k = torch.zeros((1, 2, 64, 128), dtype=torch.int8)
    s = torch.zeros((1, 2, 4))
    with pytest.raises(ValueError):
        ad.KV8Cache(k, k, s, s, 16)                                    # not on a GPU
    with pytest.raises(TypeError):
        ad.KV8Cache(k.to(torch.bfloat16), k, s, s, 16)
    with pytest.raises(ValueError):
        ad.KV8Cache(k[..., :64], k, s, s, 16)
    with pytest.raises(ValueError):
        ad.KV8Cache(k, k, s, s, 24)


def test_struct_matches_the_headers_order():
    import re
    with open(ad.HEADER_PATH) as f:
        body = re.search(r"typedef struct \{(.*?)\} adamas_kv8_cache;", f.read(), re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = [re.split(r"[\s*]+", x.strip())[-1] for x in body.split(";") if x.strip()]
    assert names == [n for n, _ in _CCache._fields_]
    assert ctypes.sizeof(_CCache) == 6 * 8 + 2 * 8 + 8 * 4


def test_helpers_pages_round_trip():
    c = Case(2, 3, 70, page=32, block=16, seed=1)
    assert np.array_equal(c._seq(c._pages(c.k, 32, 0.0)), c.k)
    assert np.array_equal(c._seq(c._pages(c.ks, 2, 1.0)), c.ks)
