"""Measured cases of the 8-bit cache operators: what each computes in plain torch
operations, the same from its definition in float64, and the framework's calls.

An 8-bit cache holds K and V rows of 128 values in e4m3 or int8 with one power-of-two
float32 scale per block of `block` positions and kv head.  Operators:

  append   new rows are quantised into the cache at each sequence's end (a block that
           already holds rows keeps a scale at least as large, and its rows are rounded
           to a larger one), then the touched window is read back as values
  dense    single-token attention over every cached position of each sequence,
           optionally adding each position's attention weight to a running sum
  sparse   the same over given positions (per query head, or one list per kv head)
  evict    the cache is shortened to `budget` rows: the first `sink`, the last `recent`
           and the largest running weights between; rows, scales and sums move along

`own` is set from outside: False runs the plain forms, True the framework's calls.
"""
import math

import torch

own = False

D = 128                       # head dimension
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
QT = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


# ------------------------------------------------------------------------- cases
def listed():
    return [
        # a 32K prompt of one sequence enters an empty cache; K and V arrive as slices of
        # a token-major projection (strided by head)
        dict(name="append_prompt_32k", op="append", B=1, Hkv=8, n=32768, start=0, ragged=False,
             Lmax=32896, page=0, block=64, fmt="e4m3", dt="bf16", codes=False),
        # one decode step of a batch: one token per sequence, in the middle of a page
        dict(name="append_step_b32_paged", op="append", B=32, Hkv=8, n=1, start=1900, ragged=True,
             Lmax=2048, page=16, block=16, fmt="e4m3", dt="bf16", codes=False),
        # ragged chunks of prompts with the keys' 2-bit codes, fp32 rows, int8 cache
        dict(name="append_chunk_b8_codes", op="append", B=8, Hkv=4, n=513, start=1000, ragged=True,
             Lmax=2048, page=0, block=32, fmt="int8", dt="f32", codes=True),
        # a short chat: latency
        dict(name="dense_1000", op="dense", B=1, Hq=32, Hkv=8, L=1000, ragged=False, page=0,
             block=64, fmt="e4m3", dt="bf16", weights=False, tail=24),
        # the 32K layer, dense (layers where sparsity is switched off)
        dict(name="dense_32k", op="dense", B=1, Hq=32, Hkv=8, L=32768, ragged=False, page=0,
             block=64, fmt="e4m3", dt="bf16", weights=False, tail=0),
        # a served batch of unequal sequences (one empty, one of a single token) over pages,
        # 8 heads per kv head, fp32 queries, weights kept for eviction
        dict(name="dense_ragged_paged_w", op="dense", B=17, Hq=32, Hkv=4, L=8191, ragged=True,
             page=16, block=16, fmt="int8", dt="f32", weights=True, tail=0),
        # 32 kv heads at 128K: the largest
        dict(name="dense_mha_128k_w", op="dense", B=1, Hq=32, Hkv=32, L=131072, ragged=False, page=0,
             block=128, fmt="e4m3", dt="bf16", weights=True, tail=0),
        # the 32K layer at budget 128: latency
        dict(name="sparse_32k_k128", op="sparse", B=1, Hq=32, Hkv=8, L=32768, k=128, ragged=False,
             shared=False, page=0, block=64, fmt="e4m3", dt="bf16", weights=False),
        # batch 8 at 32K and budget 1024, weights kept for eviction
        dict(name="sparse_b8_32k_k1024_w", op="sparse", B=8, Hq=32, Hkv=8, L=32768, k=1024,
             ragged=False, shared=False, page=0, block=64, fmt="e4m3", dt="bf16", weights=True),
        # one list per kv head over pages, some sequences shorter than the list
        dict(name="sparse_shared_paged", op="sparse", B=5, Hq=64, Hkv=8, L=5000, k=777, ragged=True,
             shared=True, page=32, block=32, fmt="int8", dt="f32", weights=False),
        # a 32K cache cut to a quarter
        dict(name="evict_32k_8k", op="evict", B=1, Hkv=8, L=32768, budget=8192, sink=4, recent=1024,
             ragged=False, page=0, block=64, fmt="e4m3"),
        # a batch of unequal sequences over pages, some shorter than the budget
        dict(name="evict_b16_paged", op="evict", B=16, Hkv=8, L=16001, budget=6000, sink=1, recent=333,
             ragged=True, page=16, block=16, fmt="int8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "dense", "sparse", "evict"])
    block = rng.choice([8, 16, 32, 64, 128])
    page = rng.choice([0, 0, block, 2 * block])
    fmt = rng.choice(["e4m3", "e4m3", "int8"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    B = _log(rng, 1, 32)
    Hkv = rng.choice([1, 2, 4, 8, 16])
    if op == "append":
        n = _log(rng, 1, max(1, 200000 // (B * Hkv)))
        start = rng.choice([0, rng.randint(1, 3000)])
        codes = page == 0 and rng.random() < 0.4
        cap = -(-(start + n + 2 * block) // max(block, page)) * max(block, page)
        return dict(op=op, B=B, Hkv=Hkv, n=n, start=start, ragged=rng.random() < 0.6, Lmax=cap,
                    page=page, block=block, fmt=fmt, dt=dt, codes=codes)
    G = rng.choice([1, 2, 4, 8])
    L = _log(rng, 1, max(2, min(262144, 2000000 // (B * Hkv))))
    ragged = B > 1 and rng.random() < 0.7
    if op == "dense":
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, L=L, ragged=ragged, page=page, block=block,
                    fmt=fmt, dt=dt, weights=rng.random() < 0.5, tail=rng.choice([0, rng.randint(1, 500)]))
    if op == "sparse":
        k = min(L, _log(rng, 1, 2048))
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, L=L, k=k, ragged=ragged,
                    shared=rng.random() < 0.4, page=page, block=block, fmt=fmt, dt=dt,
                    weights=rng.random() < 0.5)
    budget = max(1, int(L * rng.uniform(0.1, 1.1)))
    sink = rng.randint(0, min(4, budget // 2))
    recent = rng.randint(0, (budget - sink) // 2 + 1) if budget > sink else 0
    return dict(op=op, B=B, Hkv=Hkv, L=L, budget=budget, sink=sink, recent=min(recent, budget - sink),
                ragged=ragged, page=page, block=block, fmt=fmt)


def work(case):
    B, Hkv = case["B"], case["Hkv"]
    e = 4 if case.get("dt") == "f32" else 2
    op = case["op"]
    if op == "append":
        # rows in, 8-bit rows and the window's values out
        n = case["n"] // 2 + 1 if case["ragged"] else case["n"]
        W = _window(case)
        rows = B * Hkv * n
        by = 2 * rows * D * (e + 1) + 2 * B * Hkv * W * D * 2
        by += rows * D // 4 if case["codes"] else 0
        return {"bytes": by, "flops": 4 * rows * D}
    L = case["L"] // 2 + 1 if case["ragged"] else case["L"]
    if op == "evict":
        n = min(L, case["budget"])
        # weights in, kept weights out; kept 8-bit rows in and out, their values out
        return {"bytes": 4 * B * Hkv * (L + n) + 2 * B * Hkv * n * D * (2 + 2), "flops": 0}
    Hq = case["Hq"]
    io = B * Hq * D * (e + 4)
    if op == "dense":
        by = 2 * B * Hkv * L * (D + 4 / case["block"]) + io + (8 * B * Hkv * L if case["weights"] else 0)
        return {"bytes": by, "flops": 4 * B * Hq * L * D}
    rows = B * (Hkv if case["shared"] else Hq)
    k = min(case["k"], L)
    # a row that several heads' lists hold needs to be read once
    by = min(rows * k, B * Hkv * L) * 2 * D + rows * k * 4 + io + (8 * B * Hkv * case["L"] if case["weights"] else 0)
    return {"bytes": by, "flops": 4 * B * Hq * k * D}


# ------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _channels(g):
    """Four channels ten times as large as the others, as model keys have them."""
    c = torch.ones(D, device=DEV)
    c[torch.randperm(D, generator=g, device=DEV)[:4]] = 10.0
    return c


def _lens(g, case, top):
    B = case["B"]
    if not case["ragged"]:
        return torch.full((B,), top, dtype=torch.int32, device=DEV)
    x = torch.randint(0, top + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    x[0] = top
    if B > 2:
        x[1], x[2] = 0, 1
    return x


def _scale_of(amax, fmt):
    """The smallest power of two S (at least 2^-126) with amax <= 448 S (127 S for int8)."""
    m, e = torch.frexp(amax)
    top, bits = (0.875, 9) if fmt == "e4m3" else (0.9921875, 7)
    e = torch.where(amax > 0, e - bits + (m > top), -126).clamp(min=-126)
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _round8(x, fmt):
    """x rounded to the 8-bit format's values, as the 8-bit tensor."""
    if fmt == "e4m3":
        return x.to(torch.float8_e4m3fn)
    return x.round().clamp(-127, 127).to(torch.int8)


def _quantised(x, block, fmt):
    """Rows [..., L, D] float32 (L a multiple of block) as 8-bit rows and block scales."""
    y = x.view(*x.shape[:-2], -1, block * D)
    s = _scale_of(y.abs().amax(-1), fmt)
    return _round8(y / s[..., None], fmt).view(x.shape), s


def _up(n, m):
    return -(-n // m) * m


def _make_cache(g, case, cap, lens=None):
    """Values in the cache, position by position: 8-bit rows [B,Hkv,cap,D] and block
    scales [B,Hkv,cap/block], of K and of V; zero rows past each sequence's length."""
    B, Hkv, block, fmt = case["B"], case["Hkv"], case["block"], case["fmt"]
    out = []
    ch = _channels(g)
    for _ in range(2):
        q8 = torch.empty((B, Hkv, cap, D), dtype=QT[fmt], device=DEV)
        s8 = torch.empty((B, Hkv, cap // block), device=DEV)
        for b in range(B):
            x = _randn(g, Hkv, cap, D).mul_(ch)
            # token norms vary, so that blocks have different scales
            x *= torch.exp2(torch.randint(-1, 2, (Hkv, cap, 1), generator=g, device=DEV).float())
            if lens is not None:
                x *= (torch.arange(cap, device=DEV) < lens[b])[None, :, None]
            q8[b], s8[b] = _quantised(x, block, fmt)
        out += [q8, s8]
    return out


def _into_pages(g, case, cap, parts):
    """The same rows and scales in shuffled pages: K, scales, V, scales, block table."""
    B, Hkv, page, block = case["B"], case["Hkv"], case["page"], case["block"]
    nb = cap // page
    table = torch.randperm(B * nb, generator=g, device=DEV).to(torch.int32).view(B, nb)
    res = []
    for x, w in zip(parts, (page, page // block) * 2):
        y = x.view(B, Hkv, nb, w, *x.shape[3:]).transpose(1, 2).flatten(0, 1).contiguous()
        z = torch.empty_like(y)
        z.view(torch.uint8)[table.view(-1).long()] = y.view(torch.uint8)
        res.append(z)
    return res + [table]


def _cache_state(g, case, cap, lens=None, empty=False):
    block, fmt = case["block"], case["fmt"]
    if empty:
        z = torch.zeros((case["B"], case["Hkv"], cap, D), dtype=torch.uint8, device=DEV)
        s = torch.zeros((case["B"], case["Hkv"], cap // block), device=DEV)
        parts = [z.view(QT[fmt]), s, z.clone().view(QT[fmt]), s.clone()]
    else:
        parts = _make_cache(g, case, cap, lens)
    table = None
    if case["page"]:
        *parts, table = _into_pages(g, case, cap, parts)
    return dict(k=parts[0], ks=parts[1], v=parts[2], vs=parts[3], table=table, cap=cap)


def _window(case):
    return _up(case["n"] + case["block"], case["block"])


def _cap(case, L):
    return _up(max(L, 1), max(case["block"], case["page"]))


def prepare(case, seed):
    g = _gen(seed)
    B, Hkv, op = case["B"], case["Hkv"], case["op"]
    s = dict(case=case)
    if op == "append":
        n, block = case["n"], case["block"]
        starts = _lens(g, case, case["start"])
        counts = torch.full((B,), n, dtype=torch.int32, device=DEV)
        if case["ragged"]:
            counts = torch.randint(1, n + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
            counts[0] = n
        s.update(_cache_state(g, case, case["Lmax"], starts), starts=starts, counts=counts,
                 first=starts // block * block)
        x = _randn(g, B, n, 2 * Hkv, D) * _channels(g)
        if case["codes"]:
            x = (x * 16).round() / 16      # sums of 128 exact in float32: no code on a border
            s["codes"] = torch.zeros((B, Hkv, case["Lmax"], D // 4), dtype=torch.uint8, device=DEV)
            s["t"] = 0.5 * math.sqrt((124 + 400) / 128)
        x = x.to(DT[case["dt"]]).transpose(1, 2)
        s["kn"], s["vn"] = x[:, :Hkv], x[:, Hkv:]
    elif op == "evict":
        cap, dcap = _cap(case, case["L"]), _cap(case, case["budget"])
        lens = _lens(g, case, case["L"])
        s.update(_cache_state(g, case, cap, lens), lens=lens)
        # sums of softmax weights: most positions hardly ever attended, many exactly never
        w = torch.exp(3 * _randn(g, B, Hkv, cap) - 8)
        w *= torch.rand(B, Hkv, cap, generator=g, device=DEV) < 0.6
        s["w"] = w * (torch.arange(cap, device=DEV) < lens[:, None, None])
        s["dst"] = _cache_state(g, case, dcap, empty=True)
        s["w_out"] = torch.zeros((B, Hkv, dcap), device=DEV)
    else:
        Hq, L = case["Hq"], case["L"]
        cap = _cap(case, L + case.get("tail", 0))
        lens = _lens(g, case, L)
        s.update(_cache_state(g, case, cap), lens=lens)
        s["q"] = _randn(g, B, Hq, D).to(DT[case["dt"]])
        if case["weights"]:
            s["w"] = torch.rand((B, Hkv, cap), generator=g, device=DEV)
            s["w_out"] = s["w"].clone()
        if op == "sparse":
            k, rows = case["k"], Hkv if case["shared"] else Hq
            u = torch.rand((B, rows, cap), generator=g, device=DEV)
            u = u.masked_fill_(torch.arange(cap, device=DEV) >= lens[:, None, None], -1.0)
            u, i = u.topk(k, dim=-1)
            i = i.masked_fill(u < 0, cap).sort(dim=-1).values
            s["idx"] = i.masked_fill(i == cap, -1).to(torch.int32)
    if own:
        _handles(s)
    return s


def _handles(s):
    """The framework's cache objects, workspaces and prepared calls that a serving loop keeps."""
    import token_level_sparse_fwht_b200 as ad
    case = s["case"]
    B, Hkv = case["B"], case["Hkv"]

    def cache(c):
        return ad.KV8Cache(c["k"], c["v"], c["ks"], c["vs"], case["block"], codes=c.get("codes"),
                           block_table=c["table"], max_seq_len=c["cap"])

    kv = cache(s)
    if case["op"] == "append":
        ws = ad.kv8_workspace()
        W = _window(case)
        s["out"] = [torch.empty((B, Hkv, W, D), dtype=torch.bfloat16, device=DEV) for _ in "kv"]
        s["calls"] = [ad.PreparedKV8Append(kv, s["kn"], s["vn"], s["starts"], ws, counts=s["counts"],
                                           t=s.get("t")),
                      ad.PreparedKV8Read(kv, s["first"], W, *s["out"], ws)]
    elif case["op"] == "evict":
        ws = ad.kv8_workspace()
        n = case["budget"]
        dst = cache(s["dst"])
        s["keep"] = torch.empty((B, Hkv, n), dtype=torch.int32, device=DEV)
        s["lens_out"] = torch.empty_like(s["lens"])
        zero = torch.zeros_like(s["lens"])
        s["out"] = [torch.empty((B, Hkv, n, D), dtype=torch.bfloat16, device=DEV) for _ in "kv"]
        s["calls"] = [ad.PreparedKV8Evict(kv, dst, s["w"], s["w_out"], s["lens"], s["lens_out"],
                                          s["keep"], n, case["sink"], case["recent"], ws),
                      ad.PreparedKV8Read(dst, zero, n, *s["out"], ws)]
    else:
        Hq = case["Hq"]
        s["out"] = torch.empty((B, Hq, D), dtype=torch.float32, device=DEV)
        more = dict(weights=s["w"], weights_out=s["w_out"]) if case["weights"] else {}
        if case["op"] == "dense":
            ws = ad.kv8_attention_workspace(B, Hq, Hkv, s["cap"], weights=case["weights"])
            s["calls"] = [ad.PreparedKV8Attention(s["q"], kv, s["lens"], ws, s["out"], **more)]
        else:
            ws = ad.kv8_sparse_attention_workspace(B, Hq, Hkv, case["k"], shared=case["shared"],
                                                   weights=case["weights"])
            s["calls"] = [ad.PreparedKV8SparseAttention(s["q"], kv, s["idx"], ws, s["out"],
                                                        shared=case["shared"], **more)]


# --------------------------------------------------------------------------- run
def run(s):
    case = s["case"]
    if own:
        for call in s["calls"]:
            call()
        if case["op"] == "append":
            return dict(k=s["out"][0], v=s["out"][1], codes=s.get("codes"))
        if case["op"] == "evict":
            return dict(k=s["out"][0], v=s["out"][1], keep=s["keep"], lens=s["lens_out"], w=s["w_out"])
        return dict(out=s["out"], w=s.get("w_out"))
    return {"append": _append, "dense": _dense, "sparse": _sparse, "evict": _evict}[case["op"]](s)


def _seq(x, table):
    """Pages [P,Hkv,w,...] as sequences [B,Hkv,nb*w,...]; contiguous tensors as they are."""
    if table is None:
        return x
    y = x.view(torch.uint8)[table.long()].view(x.dtype)          # [B, nb, Hkv, w, ...]
    y = y.transpose(1, 2)
    return y.reshape(y.shape[0], y.shape[1], y.shape[2] * y.shape[3], *y.shape[4:])


def _values(x, sc, block):
    return (x.float().unflatten(2, (-1, block)) * sc[..., None, None]).flatten(2, 3)


def _put(x, table, rows, at, w):
    """Writes rows [B,Hkv,n,...] at sequence positions at [B,n] of x (w rows to a page)."""
    B, Hkv, n = rows.shape[:3]
    h = torch.arange(Hkv, device=DEV)[None, :, None]
    if table is None:
        b = torch.arange(B, device=DEV)[:, None, None]
        x[b, h, at[:, None]] = rows
    else:
        p = torch.gather(table.long(), 1, at // w)[:, None]
        x[p, h, (at % w)[:, None]] = rows


def _get(x, table, at, w):
    Hkv = x.shape[1]
    h = torch.arange(Hkv, device=DEV)[None, :, None]
    if table is None:
        return x[torch.arange(at.shape[0], device=DEV)[:, None, None], h, at[:, None]]
    return x[torch.gather(table.long(), 1, at // w)[:, None], h, (at % w)[:, None]]


def _append_one(s, x8, sc, new):
    case = s["case"]
    block, fmt, table = case["block"], case["fmt"], s["table"]
    W, page = _window(case), case["page"]
    at = s["first"].long()[:, None] + torch.arange(W, device=DEV)             # [B, W]
    bat = at[:, ::block] // block                                             # blocks
    inside = at < s["cap"]
    at, bat = at.clamp(max=s["cap"] - 1), bat.clamp(max=s["cap"] // block - 1)
    i = at - s["starts"].long()[:, None]
    is_new = ((i >= 0) & (i < s["counts"][:, None]) & inside)[:, None]        # [B, 1, W]
    x = torch.gather(new.float(), 2, i.clamp(0, case["n"] - 1)[:, None, :, None].expand(
        -1, case["Hkv"], -1, D)) * is_new[..., None]
    nb = W // block
    amax = x.abs().amax(-1).unflatten(2, (nb, block)).amax(-1)
    old = _get(sc, table, bat, page // block if page else 0)                  # [B, Hkv, nb]
    had = (bat * block < s["starts"][:, None])[:, None]
    touched = is_new.unflatten(2, (nb, block)).any(-1)
    scale = torch.where(touched, torch.maximum(_scale_of(amax, fmt), old * had), old)
    o8 = _get(x8.view(torch.uint8), table, at, page).view(x8.dtype)
    per = lambda t: t.repeat_interleave(block, 2)[..., None]  # noqa: E731
    kept = _round8(o8.float() * (per(old) / per(scale)).nan_to_num(1.0, 1.0, 1.0), fmt)
    behind = (i >= 0)[:, None, :, None]           # rows behind the new ones stay as they are
    y = torch.where(is_new[..., None], _round8(x / per(scale), fmt).view(torch.uint8),
                    torch.where(behind, o8.view(torch.uint8), kept.view(torch.uint8))).view(x8.dtype)
    _put(x8.view(torch.uint8), table, y.view(torch.uint8), at, page)
    _put(sc, table, scale, bat, page // block if page else 0)
    return (y.float() * per(scale)).to(torch.bfloat16)


def _hadamard():
    i = torch.arange(D, device=DEV)
    x = i[:, None] & i[None, :]
    par = (x[..., None] >> torch.arange(7, device=DEV) & 1).sum(-1) & 1
    return 1.0 - 2.0 * par.double()


def _append(s):
    k = _append_one(s, s["k"], s["ks"], s["kn"])
    v = _append_one(s, s["v"], s["vs"], s["vn"])
    if "codes" not in s:
        return dict(k=k, v=v, codes=None)
    case, n = s["case"], s["case"]["n"]
    y = s["kn"].double() @ _hadamard() / math.sqrt(D)
    t = float(torch.tensor(s["t"], dtype=torch.float32))
    c = (y >= -t).int() + (y >= 0).int() + (y >= t).int()
    c = (c.unflatten(-1, (-1, 4)) << torch.tensor([0, 2, 4, 6], device=DEV)).sum(-1).to(torch.uint8)
    i = torch.arange(case["Lmax"], device=DEV) - s["starts"].long()[:, None]  # [B, Lmax]
    is_new = ((i >= 0) & (i < s["counts"][:, None]))[:, None, :, None]
    c = torch.gather(c, 2, i.clamp(0, n - 1)[:, None, :, None].expand(-1, case["Hkv"], -1, D // 4))
    s["codes"].copy_(torch.where(is_new, c, s["codes"]))
    return dict(k=k, v=v, codes=s["codes"])


def _softmax(x, ok):
    """Softmax over the last axis where ok; rows with nothing left are zero."""
    x = x.masked_fill(~ok, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    return p / p.sum(-1, keepdim=True).clamp(min=1e-30)


def _dense(s):
    case = s["case"]
    B, Hkv, Hq = case["B"], case["Hkv"], case["Hq"]
    K = _values(_seq(s["k"], s["table"]), _seq(s["ks"], s["table"]), case["block"])
    q = s["q"].float().view(B, Hkv, Hq // Hkv, D)
    ok = (torch.arange(s["cap"], device=DEV) < s["lens"][:, None])[:, None, None]
    p = _softmax(q @ K.transpose(-1, -2) / math.sqrt(D), ok)
    del K
    V = _values(_seq(s["v"], s["table"]), _seq(s["vs"], s["table"]), case["block"])
    out = (p @ V).view(B, Hq, D)
    return dict(out=out, w=s["w"] + p.sum(2) if case["weights"] else None)


def _sparse(s):
    case = s["case"]
    B, Hkv, Hq, block = case["B"], case["Hkv"], case["Hq"], case["block"]
    R = s["idx"].shape[1]                                                     # lists per sequence
    ok = s["idx"] >= 0
    at = s["idx"].clamp(min=0).long()
    h = (torch.arange(R, device=DEV) // (R // Hkv))[None, :, None]
    if s["table"] is None:
        page, row, srow = torch.arange(B, device=DEV)[:, None, None], at, at // block
    else:
        w = case["page"]
        page = torch.gather(s["table"].long(), 1, (at // w).flatten(1)).view_as(at)
        row, srow = at % w, at % w // block
    rows = lambda x, sc: (x.view(torch.uint8)[page, h, row].view(x.dtype).float()  # noqa: E731
                          * sc[page, h, srow][..., None])
    q = s["q"].float().view(B, R, Hq // R, D)
    p = _softmax(q @ rows(s["k"], s["ks"]).transpose(-1, -2) / math.sqrt(D), ok[:, :, None])
    out = (p @ rows(s["v"], s["vs"])).view(B, Hq, D)
    if not case["weights"]:
        return dict(out=out, w=None)
    p = p.sum(2).view(B, Hkv, -1)
    return dict(out=out, w=s["w"].scatter_add(2, at.view(B, Hkv, -1), p))


def _evict(s):
    case = s["case"]
    n, sink, recent, block = case["budget"], case["sink"], case["recent"], case["block"]
    cap, dcap = s["cap"], s["dst"]["cap"]
    at = torch.arange(cap, device=DEV)
    lens = s["lens"][:, None, None].long()
    w = torch.where(s["w"].isnan(), -math.inf, s["w"])
    w = torch.where((at < sink) | (at >= lens - recent), math.inf, w)
    w = torch.where(lens <= n, 1.0, w).masked_fill(at >= lens, -math.inf)
    first = torch.where(at < lens, 0, 1).expand_as(w)
    # order by (inside the sequence, weight descending, position ascending)
    order = torch.argsort(w, dim=-1, descending=True, stable=True)
    order = order.gather(-1, torch.argsort(first.gather(-1, order), dim=-1, stable=True))[..., :n]
    new_lens = lens.clamp(max=n)
    m = order.shape[-1]
    order = order.masked_fill(torch.arange(m, device=DEV) >= new_lens, cap).sort(-1).values
    keep = torch.full((*order.shape[:2], n), -1, dtype=torch.int32, device=DEV)
    keep[..., :m] = order.masked_fill(order == cap, -1).to(torch.int32)
    ok = keep >= 0
    src = keep.clamp(min=0).long()
    res = []
    pad = _up(n, block)
    for x, sc in ((s["k"], s["ks"]), (s["v"], s["vs"])):
        y = _values(_seq(x, s["table"]), _seq(sc, s["table"]), block)
        y = torch.gather(y, 2, src[..., None].expand(-1, -1, -1, D)) * ok[..., None]
        z = torch.zeros((*y.shape[:2], pad, D), device=DEV)
        z[:, :, :n] = y
        q8, s8 = _quantised(z, block, case["fmt"])
        res.append(_values(q8, s8, block)[:, :, :n].to(torch.bfloat16))
    w = torch.zeros((*keep.shape[:2], dcap), device=DEV)
    w[..., :n] = torch.gather(s["w"], 2, src) * ok
    return dict(k=res[0], v=res[1], keep=keep, lens=new_lens.view(-1).to(torch.int32), w=w)


# ------------------------------------------------------------------------- exact
# The same outputs from the definitions in float64, by other means than above.
def _two(e):
    """2^e for whole numbers e, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _scale64(a, fmt):
    top = 448.0 if fmt == "e4m3" else 127.0
    e = torch.floor(torch.log2(a.clamp(min=1e-300) / top))
    e = torch.where(a <= top * _two(e), e, e + 1)
    e = torch.where(a <= top * _two(e), e, e + 1).clamp(min=-126)
    return _two(e)


def _near64(x, fmt):
    """Nearest value of the format, ties to even."""
    if fmt == "int8":
        return torch.round(x).clamp(-127, 127)
    mag = x.abs().clamp(min=1e-300)
    e = torch.floor(torch.log2(mag))
    e = torch.where(_two(e) > mag, e - 1, e)
    e = torch.where(_two(e + 1) <= mag, e + 1, e).clamp(min=-6)
    step = _two(e - 3)
    return torch.round(x / step) * step


def _rows64(s, x, sc):
    """All positions' values in float64, [B, Hkv, cap, D], page by page."""
    case = s["case"]
    block = case["block"]
    v = x.to(torch.float64).reshape(*x.shape[:2], -1, block, D) * sc.double()[..., None, None]
    v = v.reshape(*x.shape[:2], -1, D)
    if s["table"] is None:
        return v
    return v[s["table"].long()].permute(0, 2, 1, 3, 4).reshape(case["B"], case["Hkv"], -1, D)


def exact(case, seed):
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    B, Hkv, op, fmt, block = case["B"], case["Hkv"], case["op"], case["fmt"], case["block"]
    if op == "append":
        res = []
        W = _window(case)
        for x8, sc, new in ((s["k"], s["ks"], s["kn"]), (s["v"], s["vs"], s["vn"])):
            seq8 = _seq(x8, s["table"]).double()
            out = torch.zeros((B, Hkv, W, D), dtype=torch.float64, device=DEV)
            scs = _seq(sc, s["table"]).double()
            for b in range(B):
                st, c, f = int(s["starts"][b]), int(s["counts"][b]), int(s["first"][b])
                end = min(f + W, s["cap"])
                o = seq8[b, :, f:end].reshape(Hkv, -1, block, D)
                old = scs[b, :, f // block:end // block, None, None]
                pos = torch.arange(f, end, device=DEV).view(-1, block)
                new_rows = torch.zeros((Hkv, end - f, D), dtype=torch.float64, device=DEV)
                new_rows[:, st - f:st - f + c] = new[b, :, :c].double()
                new_rows = new_rows.view(Hkv, -1, block, D)
                fresh = (pos >= st) & (pos < st + c)
                a = new_rows.abs().amax((-1, -2), keepdim=True)
                sc_new = _scale64(a, fmt)
                held = (pos[:, :1] < st)[None, :, :, None]
                sc_new = torch.where(held, torch.maximum(sc_new, old), sc_new)
                sc_new = torch.where(fresh.any(-1)[None, :, None, None], sc_new, old)
                was_rows = torch.where(sc_new == old, o, _near64(o * old / sc_new, fmt))
                was_rows = torch.where((pos < st)[None, ..., None], was_rows, o)
                y = torch.where(fresh[None, ..., None], _near64(new_rows / sc_new, fmt), was_rows)
                out[b, :, :end - f] = (y * sc_new).reshape(Hkv, -1, D)
            res.append(out)
        return dict(k=res[0], v=res[1], codes=None)
    if op == "evict":
        n, sink, recent = case["budget"], case["sink"], case["recent"]
        dcap = s["dst"]["cap"]
        pad = _up(n, block)
        kv = [torch.zeros((B, Hkv, n, D), dtype=torch.float64, device=DEV) for _ in "kv"]
        w_out = torch.zeros((B, Hkv, dcap), dtype=torch.float64, device=DEV)
        src = [_rows64(s, s["k"], s["ks"]), _rows64(s, s["v"], s["vs"])]
        for b in range(B):
            L = int(s["lens"][b])
            w = s["w"][b, :, :L].double()
            for h in range(Hkv):
                if L <= n:
                    sel = torch.arange(L, device=DEV)
                else:
                    mid = n - sink - recent
                    o = torch.sort(w[h, sink:L - recent], descending=True, stable=True).indices[:mid] + sink
                    sel = torch.cat([torch.arange(sink, device=DEV), o.sort().values,
                                     torch.arange(L - recent, L, device=DEV)])
                w_out[b, h, :sel.numel()] = w[h][sel]
                for i in range(2):
                    y = torch.zeros((pad, D), dtype=torch.float64, device=DEV)
                    y[:sel.numel()] = src[i][b, h][sel]
                    y = y.view(-1, block * D)
                    sc = _scale64(y.abs().amax(-1, keepdim=True), fmt)
                    kv[i][b, h] = (_near64(y / sc, fmt) * sc).view(pad, D)[:n]
        return dict(k=kv[0], v=kv[1], keep=None, lens=None, w=w_out)
    Hq = case["Hq"]
    G = Hq // Hkv
    out = torch.zeros((B, Hq, D), dtype=torch.float64, device=DEV)
    w = s["w"].double().clone() if case["weights"] else None
    q = s["q"].double()
    lists = s.get("idx")
    for b in range(B):
        sub = dict(s, case=dict(case, B=1))
        cut = (lambda x: x[b:b + 1]) if s["table"] is None else (lambda x: x)
        sub["table"] = None if s["table"] is None else s["table"][b:b + 1]
        K = _rows64(sub, cut(s["k"]), cut(s["ks"]))[0]
        V = _rows64(sub, cut(s["v"]), cut(s["vs"]))[0]
        for h in range(Hq):
            if op == "dense":
                sel = torch.arange(int(s["lens"][b]), device=DEV)
            else:
                sel = lists[b, h // G if case["shared"] else h].long()
                sel = sel[sel >= 0]
            if sel.numel() == 0:
                continue
            p = torch.softmax(K[h // G][sel] @ q[b, h] / math.sqrt(D), 0)
            out[b, h] = p @ V[h // G][sel]
            if w is not None:
                w[b, h // G].index_add_(0, sel, p)
    return dict(out=out, w=w)
