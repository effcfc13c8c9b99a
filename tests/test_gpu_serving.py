"""GPU parity of the serving operators (rotary positions and their gradient, the
paged cache written and read, attention of new tokens over it) against plain
64-bit implementations, at the sizes, strides and masks where they can go wrong."""
import math
import random

import pytest

import serving_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import attention_rank_additive_b200 as fb  # noqa: E402

F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from attention_rank_additive_b200 import build
    build.build()
    fb.lib()
    yield
    torch.cuda.synchronize()


def _status():
    return fb.fb_check_device_error(torch.cuda.current_stream().cuda_stream)


def _randn(shape, seed, dtype=torch.float32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


# ------------------------------------------------------------------- rotary

def _strided(shape, layout, seed, dtype):
    """[B, H, N, d] on the GPU: contiguous, token-major, or a slice of a wider row at an odd offset."""
    B, H, N, d = shape
    if layout == "bhnd":
        return _randn(shape, seed, dtype).cuda()
    if layout == "bnhd":
        return _randn((B, N, H, d), seed, dtype).cuda().transpose(1, 2)
    wide = _randn((B, N, H, d + 7), seed, dtype).cuda()
    return wide[..., 3:3 + d].transpose(1, 2)


ROPE = [  # dtype, B, Hq, Hk, N, d, rot, interleaved, layout, first position
    (torch.bfloat16, 1, 1, 1, 1, 64, 64, False, "bhnd", 0),
    (torch.bfloat16, 2, 12, 12, 1, 64, 64, False, "bnhd", 2047),
    (torch.bfloat16, 3, 4, 2, 37, 128, 64, True, "bnhd", 999983),
    (torch.bfloat16, 2, 6, 1, 130, 80, 20, False, "bhnd", 7),
    (torch.bfloat16, 1, 3, 3, 5, 96, 24, True, "odd", 100000),
    (torch.float32, 2, 5, 5, 33, 48, 48, True, "bhnd", 0),
    (torch.float32, 1, 8, 2, 700, 128, 32, False, "bnhd", 524288),
    (torch.float32, 2, 3, 2, 9, 33, 22, False, "odd", 12),
    (torch.bfloat16, 1, 2, 2, 3, 2, 2, True, "bhnd", 2 ** 31 - 60),
    (torch.bfloat16, 1, 40, 8, 2500, 128, 128, False, "bnhd", 31),
]


def _rope_tol(y, x, dtype, factor):
    """One rounding of the result; angle, sine, cosine and products within 2^-21 of the pair's size."""
    size = x.abs().to(F64).amax(-1, keepdim=True) * abs(factor)
    return torch.finfo(dtype).eps / 2 * y.abs() + 2.0 ** -21 * 2 * size + 1e-40


@pytest.mark.parametrize("dtype,B,Hq,Hk,N,d,rot,inter,layout,first", ROPE)
def test_rope_and_gradient_match_reference(dtype, B, Hq, Hk, N, d, rot, inter, layout, first):
    r = fb.Rope.scaled(rot, scaling="yarn" if rot > 2 else "none", by=16.0, interleaved=inter)
    q, k = _strided((B, Hq, N, d), layout, 1, dtype), _strided((B, Hk, N, d), layout, 2, dtype)
    pos = (torch.arange(N)[None] + first + torch.arange(B)[:, None] * 3).to(torch.int32)
    for call, sign in ((fb.rope, 1.0), (fb.rope_bwd, -1.0)):
        out = call(q, k, r, pos.cuda())
        torch.cuda.synchronize()
        for x, y in zip((q, k), out):
            assert y.shape == x.shape and y.dtype == dtype
            want = ref.rope(x.cpu(), r.frequencies, pos, rot, inter, r.factor, sign)
            err = (y.cpu().to(F64) - want).abs()
            tol = _rope_tol(want, x.cpu(), dtype, r.factor)
            assert (err <= tol).all(), (err / tol).max()
            if rot < d:
                assert torch.equal(y[..., rot:], x[..., rot:])
    assert _status() == fb.FB_OK


def test_rope_gradient_is_the_adjoint_and_the_difference():
    """rope is linear in x: <rope(x), g> = <x, rope_bwd(g)>, and its difference along any direction is rope of it."""
    r = fb.Rope.scaled(40, interleaved=False, factor=1.25)
    x, g, h = (_randn((2, 3, 50, 64), s).cuda() for s in (1, 2, 3))
    pos = torch.arange(50, dtype=torch.int32, device="cuda") * 17
    y, _ = fb.rope(x, None, r, pos)
    dx, _ = fb.rope_bwd(g, None, r, pos)
    a, b = (y.double() * g.double()).sum(), (x.double() * dx.double()).sum()
    assert abs(a - b) <= 2.0 ** -20 * (y.double().abs() * g.double().abs()).sum()
    step = 0.5
    y2, _ = fb.rope(x + step * h, None, r, pos)
    dirs = ((y2.double() - y.double()) * g.double()).sum() / step
    want = (h.double() * dx.double()).sum()
    assert abs(dirs - want) <= 2.0 ** -18 * ((y2.double().abs() + y.double().abs()) * g.double().abs()).sum() / step


def test_rope_in_place_default_positions_and_shared_ones():
    r = fb.Rope.scaled(32)
    q, k = _randn((3, 4, 9, 64), 1, torch.bfloat16).cuda(), _randn((3, 2, 9, 64), 2, torch.bfloat16).cuda()
    want = fb.rope(q, k, r)
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    for p in (pos, pos[None], pos[None].repeat(3, 1), pos[None].expand(3, 9)):
        assert all(torch.equal(a, b) for a, b in zip(want, fb.rope(q, k, r, p)))
    q2, k2 = q.clone(), k.clone()
    got = fb.rope(q2, k2, r, pos, out=(q2, k2))
    assert got[0] is q2 and all(torch.equal(a, b) for a, b in zip(want, got))
    # a prompt turned in one call and token by token agree to the bit
    for n in range(9):
        one = fb.rope(q[:, :, n:n + 1], k[:, :, n:n + 1], r, pos[n:n + 1])
        assert all(torch.equal(a[:, :, n:n + 1], b) for a, b in zip(want, one))


# -------------------------------------------------------------------- cache

def _cache(pages, H, page, d, kind, seed):
    k, v = _randn((pages, H, page, d), seed), _randn((pages, H, page, d), seed + 1)
    if kind == "bf16":
        return fb.PagedCache(k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda())
    (kc, ks), (vc, vs) = ref.quantise(k), ref.quantise(v * torch.exp2(_randn((pages, H, page, 1), seed + 2).round()))
    return fb.PagedCache(kc.view(torch.float8_e4m3fn).cuda(), vc.view(torch.float8_e4m3fn).cuda(),
                         ks.cuda(), vs.cuda())


def _table(B, per, total, seed):
    rng = random.Random(seed)
    order = list(range(total))
    rng.shuffle(order)
    return torch.tensor(order[:B * per], dtype=torch.int32).view(B, per)


def _bytes(t):
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int16)


CACHE = [  # cache, dtype, B, H, N, d, page, starts, counts, layout
    ("bf16", torch.bfloat16, 1, 1, 1, 16, 16, [0], None, "bhnd"),
    ("bf16", torch.float32, 3, 2, 40, 48, 16, [0, 15, 33], [40, 0, 17], "bnhd"),
    ("e4m3", torch.bfloat16, 2, 3, 1, 128, 64, [63, 64], None, "bnhd"),
    ("e4m3", torch.float32, 2, 2, 70, 80, 32, [5, 31], [70, 1], "bhnd"),
    ("e4m3", torch.bfloat16, 4, 8, 33, 64, 256, [0, 255, 256, 7], [33, 33, 2, 0], "bnhd"),
    ("e4m3", torch.bfloat16, 1, 5, 300, 112, 128, [100], None, "bhnd"),
]


@pytest.mark.parametrize("kind,dtype,B,H,N,d,page,starts,counts,layout", CACHE)
def test_cache_write_and_read(kind, dtype, B, H, N, d, page, starts, counts, layout):
    per = -(-(max(starts) + N) // page)
    cache = _cache(B * per + 2, H, page, d, kind, 5)
    table = _table(B, per, B * per + 2, 6)
    k, v = _strided((B, H, N, d), layout, 7, dtype), _strided((B, H, N, d), layout, 8, dtype)
    k[0, 0, 0] = 0.0  # a row of zeros, one of tiny values, one with a single large one
    v[-1, -1, 0] *= 2.0 ** -130 if dtype == torch.float32 else 2.0 ** -100
    v[0, 0, 0, d // 2] = 3e38
    n = counts if counts is not None else [N] * B
    want = []
    for name, new in (("k", k), ("v", v)):
        pool = getattr(cache, name).cpu().clone()
        scale = getattr(cache, name + "_scale")
        scale = None if scale is None else scale.cpu().clone()
        if kind == "e4m3":
            codes, bytes_ = ref.quantise(new.cpu())
            pool = pool.view(torch.uint8)
        for b in range(B):
            for i in range(n[b]):
                at, place = int(table[b, (starts[b] + i) // page]), (starts[b] + i) % page
                if kind == "e4m3":
                    pool[at, :, place], scale[at, :, place] = codes[b, :, i], bytes_[b, :, i]
                else:
                    pool[at, :, place] = new[b, :, i].cpu().to(torch.bfloat16)
        want.append((pool, scale))
    dev = [None if x is None else torch.tensor(x, dtype=torch.int32).cuda() for x in (starts, counts)]
    fb.cache_write(cache, k, v, table.cuda(), *dev)
    assert _status() == fb.FB_OK
    for (pool, scale), name in zip(want, "kv"):
        assert torch.equal(_bytes(getattr(cache, name).cpu()), _bytes(pool)), name
        if scale is not None:
            assert torch.equal(getattr(cache, name + "_scale").cpu(), scale), name
    for out in (torch.bfloat16, torch.float32):
        got = fb.cache_read(cache, table.cuda(), *dev, N, dtype=out)
        assert _status() == fb.FB_OK
        for x, name in zip(got, "kv"):
            scale = getattr(cache, name + "_scale")
            values = ref.pool_values(getattr(cache, name).cpu(), None if scale is None else scale.cpu())
            full = torch.zeros(B, H, N, d, dtype=F64)
            for b in range(B):
                full[b, :, :n[b]] = ref.rows(values, table[b], starts[b], n[b])
            # 8-bit values have 4 significant bits, so bf16 holds them exactly while they are normal
            assert ((x.cpu().to(F64) - full).abs() <= 2.0 ** -133).all()


def test_cache_special_values():
    cache = fb.PagedCache.empty(1, 1, 16, 16, torch.float8_e4m3fn)
    x = torch.zeros(1, 1, 4, 16)
    x[0, 0, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 7.0])
    x[0, 0, 1, :3] = torch.tensor([448.0, -448.0, 449.0])
    x[0, 0, 2, :2] = torch.tensor([1e-45, -1e-45])
    x[0, 0, 3, :2] = torch.tensor([3.4e38, -3.4e38])
    tab = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    fb.cache_write(cache, x.cuda(), x.cuda(), tab, zero)
    codes, scale = ref.quantise(x)
    assert torch.equal(cache.k.view(torch.uint8)[0, :, :4].cpu(), codes[0])
    assert torch.equal(cache.k_scale.view(torch.uint8)[0, :, :4].cpu(), scale[0])
    k, _ = fb.cache_read(cache, tab, None, None, 4, dtype=torch.float32)
    assert k[0, 0, 0, 0] == 448 * 2.0 ** -6 and k[0, 0, 0, 2].isnan() and k[0, 0, 0, 3] == 7.0
    assert _status() == fb.FB_OK


def test_cache_bad_tables_are_skipped_and_flagged():
    cache = _cache(4, 2, 16, 64, "bf16", 1)
    before = cache.k.clone(), cache.v.clone()
    k = _randn((2, 2, 3, 64), 3, torch.bfloat16).cuda()
    start = torch.tensor([0, 40], dtype=torch.int32, device="cuda")  # the second lies past the table
    for table in ([[-1], [0]], [[4], [0]], [[2 ** 31 - 1], [0]]):
        tab = torch.tensor(table, dtype=torch.int32, device="cuda")
        fb.cache_write(cache, k, k, tab, start)
        assert _status() == fb.FB_ERR_RANGE
        assert torch.equal(cache.k, before[0]) and torch.equal(cache.v, before[1])
        got = fb.cache_read(cache, tab, start, None, 3)
        assert _status() == fb.FB_ERR_RANGE and all((x == 0).all() for x in got)
        o, lse = fb.attn_cache(k, cache, tab, start)
        assert _status() == fb.FB_ERR_RANGE and torch.isfinite(o).all()
    neg = torch.tensor([-5, -1], dtype=torch.int32, device="cuda")
    fb.cache_write(cache, k[:, :, :1], k[:, :, :1], torch.zeros(2, 1, dtype=torch.int32, device="cuda"), neg)
    assert _status() == fb.FB_ERR_RANGE and torch.equal(cache.k, before[0])
    assert _status() == fb.FB_OK


# ---------------------------------------------------------------- attention

def _tree(B, T, seed):
    rng = random.Random(seed)
    seen, depth = torch.zeros(B, T, T, dtype=torch.bool), torch.zeros(B, T, dtype=torch.int32)
    for b in range(B):
        for t in range(T):
            p = rng.randint(max(-1, t - 5), t - 1) if t else -1
            if p >= 0:
                seen[b, t] = seen[b, p]
                depth[b, t] = depth[b, p] + 1
            seen[b, t, t] = True
    return seen, depth


def _words(seen):
    B, T, _ = seen.shape
    bits = torch.zeros(B, T, -(-T // 32) * 32, dtype=torch.int64)
    bits[:, :, :T] = seen
    w = (bits.view(B, T, -1, 32) << torch.arange(32)).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def _bias(kind, Hq, H, P, seed):
    if kind == "none":
        return None, None
    pos = torch.arange(P, dtype=F64)
    if kind == "alibi":
        m = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, dtype=F64) / Hq)
        return (torch.stack([-m[:, None] * pos, m[:, None].expand(Hq, P)], -1).float(),
                torch.stack([torch.ones_like(pos), pos], -1).float()[None])
    if kind.startswith("sandwich"):
        R = int(kind[8:])
        a = pos[:, None] * 10000.0 ** (-2.0 * torch.arange(1, R // 2 + 1, dtype=F64) / R)
        phi = torch.stack([a.cos(), a.sin()], -1).reshape(1, P, R).float()
        return phi, phi
    R = int(kind[3:])  # "low17": factors of each head, columns of very different size
    size = torch.exp2(torch.linspace(-12, 12, R))
    return _randn((Hq, P, R), seed) * R ** -0.5 * size, _randn((H, P, R), seed + 1) / size


def _case(kind, d, Hq, H, T, page, prefix, counts, bias, tree, seed=0):
    B = len(prefix)
    per = max(1, -(-(max(prefix) + T) // page))
    cache = _cache(B * per + 1, H, page, d, kind, seed + 10)
    table = _table(B, per, B * per + 1, seed + 11)
    q = _randn((B, Hq, T, d), seed + 12, torch.bfloat16)
    mask = depth = None
    if tree:
        seen, depth = _tree(B, T, seed + 13)
        mask = _words(seen)
    fq, fk = _bias(bias, Hq, H, per * page, seed + 14)
    return dict(q=q, cache=cache, table=table, prefix=torch.tensor(prefix, dtype=torch.int32),
                counts=None if counts is None else torch.tensor(counts, dtype=torch.int32), mask=mask, depth=depth,
                fq=fq, fk=fk)


def _call(c, **kw):
    dev = lambda x: None if x is None else x.cuda()  # noqa: E731
    bias = None if c["fq"] is None else fb.CacheBias(c["fq"].cuda(), c["fk"].cuda())
    return fb.attn_cache(c["q"].cuda(), c["cache"], c["table"].cuda(), c["prefix"].cuda(), dev(c["counts"]),
                         tree_mask=dev(c["mask"]), depths=dev(c["depth"]), bias=bias, **kw)


def _want(c):
    cache = c["cache"]
    e4m3 = cache.k_scale is not None
    kv = ref.pool_values(cache.k.cpu(), cache.k_scale.cpu() if e4m3 else None)
    vv = ref.pool_values(cache.v.cpu(), cache.v_scale.cpu() if e4m3 else None)
    counts = c["counts"] if c["counts"] is not None else [c["q"].shape[2]] * c["q"].shape[0]
    # The roundings of a probability that the header names: fp16's half step, 2^-11 of it, where an 8-bit cache meets at
    # most 16 query rows of a key/value head; bf16's, 2^-8, in the 128-row tiles (8-bit values become bf16 there: their
    # row's power of two leaves fp16's range) and for a 16-bit cache.
    few = c["q"].shape[1] // cache.heads * c["q"].shape[2] <= 16
    return ref.attend(c["q"], kv, vv, c["table"], c["prefix"], counts, c["mask"], c["depth"], c["fq"], c["fk"],
                      part_bits=11 if e4m3 and few else 8)


def _compare(got, want):
    (o, lse), (ro, rl, to, tl) = (x.cpu().to(F64) for x in got), want
    assert torch.equal(lse == -math.inf, rl == -math.inf)
    some = rl > -math.inf
    err = (lse[some] - rl[some]).abs() / tl[some]
    assert not some.any() or err.max() <= 1.0, f"LSE: {float(err.max()):.3g} of its bound"
    assert torch.isfinite(o).all()
    over = (o - ro).abs() - to
    assert (over <= 0).all(), f"O: {float(over.max()):.3g} past its bound"


ATTEND = [  # cache, d, Hq, H, T, page, prefix, counts, bias, tree
    ("bf16", 64, 1, 1, 1, 16, [0], None, "none", False),
    ("bf16", 64, 12, 12, 1, 16, [700], None, "sandwich64", False),
    ("e4m3", 128, 16, 16, 1, 64, [1, 15, 16, 17, 127, 1023], None, "alibi", False),
    ("bf16", 128, 32, 4, 1, 128, [5000, 63], None, "none", False),
    ("e4m3", 16, 2, 1, 1, 16, [33, 0], None, "low3", False),
    ("bf16", 16, 4, 2, 3, 32, [31, 32, 33], [3, 1, 2], "low17", False),
    ("e4m3", 48, 3, 3, 24, 16, [100, 0, 511], [24, 24, 5], "alibi", True),
    ("bf16", 80, 4, 1, 5, 256, [255, 256, 1], None, "low32", True),
    ("e4m3", 96, 8, 2, 61, 64, [130, 64], [61, 33], "low8", True),
    ("bf16", 112, 6, 2, 33, 16, [47], None, "sandwich32", True),
    ("bf16", 32, 8, 8, 64, 64, [200, 3], [64, 1], "low48", True),
    ("e4m3", 64, 16, 2, 17, 32, [77, 2000], None, "sandwich128", False),
    ("e4m3", 128, 32, 4, 61, 64, [900, 31], [61, 60], "low32", True),
    ("bf16", 128, 8, 8, 1, 64, [64 * k for k in range(40)], None, "alibi", False),
    ("bf16", 64, 2, 2, 200, 16, [300, 0], [200, 150], "none", False),
]


@pytest.mark.parametrize("kind,d,Hq,H,T,page,prefix,counts,bias,tree", ATTEND)
def test_attn_cache_matches_reference(kind, d, Hq, H, T, page, prefix, counts, bias, tree):
    c = _case(kind, d, Hq, H, T, page, prefix, counts, bias, tree)
    ws = fb.cache_workspace(len(prefix), Hq, H, T, d)
    want = _want(c)
    got = _call(c, workspace=ws)
    assert _status() == fb.FB_OK
    _compare(got, want)
    again = _call(c, workspace=ws)  # the workspace is as it was, and the result the same to the bit
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("T", [4, 40])
def test_rows_that_see_nothing_and_values_that_are_not_seen(kind, T):
    """No context and an empty mask row: O = 0, LSE = -inf. Infinities and NaN in drafted rows, in the rows behind the
    last token and in unused pages stay where they are seen."""
    c = _case(kind, 64, 4, 2, T, 16, [0, 20], [T, T - 1], "low8", True, seed=3)
    mask = c["mask"]
    mask[0, 2] = 0
    seen_1 = (mask[1, :, 0] >> 1) & 1  # rows of sequence 1 that see its drafted token 1
    clean = _want(c)
    at = lambda b, i: (int(c["table"][b, i // 16]), i % 16)  # noqa: E731
    cache = c["cache"]
    for name in "kv":
        pool, scale = getattr(cache, name), getattr(cache, name + "_scale")
        used = [at(0, i) for i in range(T)] + [at(1, i) for i in range(20 + T - 1)]
        flat = torch.ones(pool.shape[0], 16, dtype=torch.bool)
        for p, i in used:
            flat[p, i] = False
        p, i = at(1, 21)
        flat[p, i] = True
        where = flat.nonzero().cuda()
        if kind == "bf16":
            pool[where[:, 0], :, where[:, 1]] = math.nan
            pool[where[:, 0], :, where[:, 1], 5] = math.inf
        else:
            pool.view(torch.uint8)[where[:, 0], :, where[:, 1]] = 0x7F
            scale.view(torch.uint8)[where[:, 0], :, where[:, 1]] = 0xFF
    o, lse = _call(c)
    ro, rl, to, tl = clean
    hit = torch.zeros(2, T, dtype=torch.bool)
    hit[1] = (seen_1 == 1) & (torch.arange(T) < T - 1)
    assert o[1].cpu()[:, hit[1]].isnan().any() if hit.any() else True
    keep = ~hit[:, None, :].expand(2, 4, T)
    o, lse = o.cpu().to(F64), lse.cpu().to(F64)
    assert (lse[0, :, 2] == -math.inf).all() and (o[0, :, 2] == 0).all()
    assert (lse[1, :, T - 1] == -math.inf).all() and (o[1, :, T - 1] == 0).all()
    assert torch.equal(lse[keep] == -math.inf, rl[keep] == -math.inf)
    some = keep & (rl > -math.inf)
    assert ((lse[some] - rl[some]).abs() <= tl[some]).all()
    assert ((o - ro).abs() <= to)[keep].all()


def test_infinite_value_reaches_the_rows_that_see_it():
    c = _case("bf16", 32, 1, 1, 3, 16, [4], None, "none", False)
    p, i = int(c["table"][0, 0]), 5  # drafted token 1: rows 1 and 2 see it
    c["cache"].v[p, 0, i, 7] = math.inf
    o, _ = _call(c)
    assert torch.isfinite(o[0, 0, 0]).all() and (o[0, 0, 1:, 7] == math.inf).all()
    o = o[0, 0, :, [j for j in range(32) if j != 7]]
    assert torch.isfinite(o).all()


def test_bias_of_the_lowest_values():
    """Factors that shut keys out with the type's lowest value, or all keys of a row: fp32 scores, so the softmax of a
    row whose scores all are -3e38 is uniform, as its definition says."""
    low = torch.finfo(torch.float32).min
    c = _case("bf16", 64, 2, 1, 1, 16, [40], None, "none", False)
    P = 48
    fk = torch.zeros(1, P, 1)
    fk[0, 10:] = 1.0
    c["fq"], c["fk"] = torch.full((2, P, 1), low), fk
    o, lse = _call(c)
    v = ref.rows(c["cache"].v.cpu().to(F64), c["table"][0], 0, 41)[0]
    c2 = _case("bf16", 64, 2, 1, 1, 16, [40], None, "none", False)
    full = _want(dict(c, fq=None, fk=None))
    del full, c2
    k = ref.rows(c["cache"].k.cpu().to(F64), c["table"][0], 0, 41)[0]
    x = (c["q"][0, :, 0].to(F64) @ k[:10].T) / 8
    want = torch.softmax(x, -1) @ v[:10]
    assert ((o[0, :, 0].cpu().to(F64) - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -7 * v[:10].abs().amax(0)).all()
    assert ((lse[0, :, 0].cpu().to(F64) - torch.logsumexp(x, -1)).abs() <= 1e-4).all()
    c["fk"] = torch.ones(1, P, 1)
    o, lse = _call(c)
    assert ((o[0, :, 0].cpu().to(F64) - v.mean(0)).abs() <= 2.0 ** -8 * v.abs().amax(0)).all()
    assert (lse < -3e38).all() and torch.isfinite(lse).all()


def test_value_rows_of_very_different_size():
    """An e4m3 row of values 2^100 larger that carries no weight does not push the others out of fp16's range."""
    c = _case("e4m3", 64, 2, 2, 1, 16, [60], None, "none", False)
    c["cache"].v_scale.view(torch.uint8)[int(c["table"][0, 0]), :, 3] = 227
    P = 64
    fk = torch.zeros(1, P, 1)
    fk[0, 3] = 1.0
    c["fq"], c["fk"] = torch.full((2, P, 1), -1e4), fk
    _compare(_call(c), _want(c))


def test_positions_past_the_factors_are_flagged():
    c = _case("bf16", 64, 1, 1, 1, 16, [30], None, "alibi", False)
    c["fq"], c["fk"] = c["fq"][:, :20].contiguous(), c["fk"][:, :20].contiguous()
    o, _ = _call(c)
    assert _status() == fb.FB_ERR_RANGE and torch.isfinite(o).all()


def test_captured_calls_on_another_stream():
    """One graph of a whole step (turn, write, attend) replayed with new inputs, beside eager calls on another stream
    with a workspace of their own."""
    B, H, T, d = 3, 4, 1, 64
    cache = _cache(13, H, 16, d, "e4m3", 1)
    table = _table(B, 4, 13, 2).cuda()
    r = fb.Rope.scaled(64)
    q, k, v = (_randn((B, T, H, d), s, torch.bfloat16).cuda() for s in (3, 4, 5))
    prefix = torch.tensor([5, 30, 62], dtype=torch.int32, device="cuda")
    pos = prefix[:, None].clone()

    def step(ws):
        qr, kr = fb.rope(q.transpose(1, 2), k.transpose(1, 2), r, pos)
        fb.cache_write(cache, kr, v.transpose(1, 2), table, prefix)
        return fb.attn_cache(qr.contiguous(), cache, table, prefix, workspace=ws)

    ws, ws2 = (fb.cache_workspace(B, H, H, T, d) for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(ws)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step(ws)
    torch.cuda.current_stream().wait_stream(side)
    for s in range(3):
        for x, seed in ((q, 10), (k, 20), (v, 30)):
            x.copy_(_randn(x.shape, seed + s, torch.bfloat16))
        if s:
            prefix.sub_(1)
            pos.sub_(1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in out]
        with torch.cuda.stream(side):
            eager = step(ws2)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, eager))
    assert _status() == fb.FB_OK


def test_decode_steps_agree_with_full_attention():
    """A run as it is used: prompt turned and written, tokens decoded one at a time with ALiBi factors, then the same
    tokens as one drafted chain, and the framework's full causal attention over what the cache holds."""
    B, Hq, H, N, d, steps = 2, 4, 4, 90, 64, 6
    total = N + steps
    r = fb.Rope.scaled(64, scaling="linear", by=4.0)
    q, k, v = (_randn((B, H, total, d), s, torch.bfloat16).cuda() for s in (1, 2, 3))
    qr, kr = fb.rope(q, k, r)
    pq, pk = fb.factors_alibi(Hq, total)
    bias = fb.CacheBias(pq, pk)
    for dtype in (torch.bfloat16, torch.float8_e4m3fn):
        cache = fb.PagedCache.empty(2 * 6 + 1, H, 16, d, dtype)
        table = _table(B, 6, 13, 4).cuda()
        at = lambda n: torch.full((B,), n, dtype=torch.int32, device="cuda")  # noqa: E731
        fb.cache_write(cache, kr[:, :, :N], v[:, :, :N], table, at(0))
        ones = []
        for n in range(N, total):
            fb.cache_write(cache, kr[:, :, n:n + 1], v[:, :, n:n + 1], table, at(n))
            ones.append(fb.attn_cache(qr[:, :, n:n + 1].contiguous(), cache, table, at(n), bias=bias))
        chain = fb.attn_cache(qr[:, :, N:].contiguous(), cache, table, at(N), bias=bias)
        kc, vc = fb.cache_read(cache, table, None, None, total)
        full = fb.attn(qr, kc, vc, pq, pk, causal=True)
        assert _status() == fb.FB_OK
        for i in range(steps):
            for a, b, c in zip(ones[i], chain, full):
                a, b, c = a[:, :, 0].double(), b[:, :, i].double(), c[:, :, N + i].double()
                # all three round probabilities (2^-8 of weights that add up to 1, on values below 5) and O
                assert (a - b).abs().max() <= 2.0 ** -6 and (a - c).abs().max() <= 2e-2


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,context", [(1, 0), (1, 5000), (6, 40), (40, 0), (40, 3000), (150, 90)])
def test_nan_is_not_taken_for_a_row_without_keys(kind, T, context):
    """A query with a NaN, and a context key with one, make their rows NaN (O and LSE), also where no other score of a
    part of the row is finite; the other rows keep their results."""
    c = _case(kind, 64, 2, 2, T, 16, [context, context], None, "none", False, seed=7)
    clean = _call(c)
    c["q"][0, 1, T - 1, 9] = math.nan
    o, lse = _call(c)
    assert o[0, 1, T - 1].isnan().all() and lse[0, 1, T - 1].isnan()
    hit = torch.zeros(2, 2, T, dtype=torch.bool, device="cuda")
    hit[0, 1, T - 1] = True
    assert torch.equal(o[~hit], clean[0][~hit]) and torch.equal(lse[~hit], clean[1][~hit])
    # new token 0's key in head 0 of sequence 1: all rows of that head see it
    pool = c["cache"].k
    at = int(c["table"][1, context // 16]), 0, context % 16, 3
    if kind == "bf16":
        pool[at] = math.nan
    else:
        pool.view(torch.uint8)[at] = 0x7F
    o, lse = _call(c)
    hit[1, 0] = True
    assert o[hit].isnan().all() and lse[hit].isnan().all()
    assert torch.equal(o[~hit], clean[0][~hit]) and torch.equal(lse[~hit], clean[1][~hit])
    assert _status() == fb.FB_OK


def test_smallest_queries_against_the_largest_scales():
    """Queries near the least normal number with 8-bit keys whose scale is the largest: the products are ordinary."""
    c = _case("e4m3", 64, 1, 1, 1, 16, [40], None, "none", False, seed=9)
    c["q"] = (c["q"].float() * 2.0 ** -124).to(torch.bfloat16)
    c["cache"].k_scale.view(torch.uint8).fill_(127 + 116)
    _compare(_call(c), _want(c))


def test_refusals():
    c = _case("bf16", 64, 4, 2, 2, 16, [20], None, "low8", True)
    cache, table, prefix, q = c["cache"], c["table"].cuda(), c["prefix"].cuda(), c["q"].cuda()
    e4 = _cache(3, 2, 16, 64, "e4m3", 1)
    ok = dict(tree_mask=c["mask"].cuda(), depths=c["depth"].cuda())
    k = torch.zeros(1, 2, 3, 64, device="cuda", dtype=torch.bfloat16)
    r = fb.Rope.scaled(64)
    refused = [
        lambda: fb.attn_cache(q.float(), cache, table, prefix, **ok),
        lambda: fb.attn_cache(q.cpu(), cache, table, prefix, **ok),
        lambda: fb.attn_cache(q[..., :32], cache, table, prefix, **ok),
        lambda: fb.attn_cache(q.transpose(1, 2).contiguous().transpose(1, 2), cache, table, prefix, **ok),
        lambda: fb.attn_cache(q, cache, table.long(), prefix, **ok),
        lambda: fb.attn_cache(q, cache, table.expand(2, -1), prefix, **ok),
        lambda: fb.attn_cache(q, cache, table, prefix.expand(2), **ok),
        lambda: fb.attn_cache(q, cache, table, prefix.cpu(), **ok),
        lambda: fb.attn_cache(q, cache, table, prefix, tree_mask=ok["tree_mask"][:, :1]),
        lambda: fb.attn_cache(q, cache, table, prefix, tree_mask=ok["tree_mask"].float()),
        lambda: fb.attn_cache(q, cache, table, prefix, depths=ok["depths"].cpu()),
        lambda: fb.attn_cache(q, cache, table, prefix, out=torch.empty_like(q).float()),
        lambda: fb.attn_cache(q, cache, table, prefix, lse=torch.empty(1, 4, 2, device="cuda", dtype=torch.bfloat16)),
        lambda: fb.attn_cache(q, cache, table, prefix, workspace=torch.zeros(64, device="cuda")),
        lambda: fb.cache_write(cache, k[:, :1], k[:, :1], table, prefix),
        lambda: fb.cache_write(cache, k, k[:, :, :2], table, prefix),
        lambda: fb.cache_write(cache, k, k.float(), table, prefix),
        lambda: fb.cache_write(cache, k.half(), k.half(), table, prefix),
        lambda: fb.cache_write(cache, k, k, table, None),
        lambda: fb.cache_read(cache, table, None, None, 4, dtype=torch.float16),
        lambda: fb.cache_read(cache, table, None, None, 4, out=(k, k)),
        lambda: fb.PagedCache(cache.k, cache.v.transpose(2, 3)),
        lambda: fb.PagedCache(cache.k, cache.v, torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")),
        lambda: fb.PagedCache(e4.k, e4.v),
        lambda: fb.PagedCache(e4.k, e4.v, e4.k_scale[:, :1], e4.v_scale),
        lambda: fb.CacheBias(torch.zeros(1, 4, 8, device="cuda"), torch.zeros(1, 5, 8, device="cuda")),
        lambda: fb.CacheBias(torch.zeros(1, 4, 8), torch.zeros(1, 4, 8)),
        lambda: fb.rope(q.half(), None, r), lambda: fb.rope(q.cpu(), None, r), lambda: fb.rope(q, k, r),
        lambda: fb.rope(q, None, r, positions=torch.zeros(3, dtype=torch.int32, device="cuda")),
        lambda: fb.rope(q, None, r, positions=torch.zeros(2, device="cuda")),
        lambda: fb.rope(q, None, r, out=(torch.empty_like(q)[..., :1].expand_as(q), None)),
        lambda: fb.rope(q.transpose(2, 3), None, r),
        lambda: fb.Rope([]), lambda: fb.Rope([1.0], factor=math.inf), lambda: fb.Rope.scaled(64, scaling="other"),
        lambda: fb.cache_workspace(1, 3, 2, 1, 64),
    ]
    for i, call in enumerate(refused):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    for call, status in (
            (lambda: fb.attn_cache(q, cache, table, prefix, scale=0.0), fb.FB_ERR_INVALID_ARG),
            (lambda: fb.attn_cache(q, cache, table, prefix, workspace=torch.zeros(256, device="cuda", dtype=torch.uint8)),
             fb.FB_ERR_WORKSPACE),
            (lambda: fb.cache_write(cache, torch.zeros(1, 2, 3, 65, device="cuda")[..., :64],
                                    torch.zeros(1, 2, 3, 65, device="cuda")[..., :64], table, prefix),
             fb.FB_ERR_UNSUPPORTED),
            (lambda: fb.rope(q[:, :, :0], None, r), fb.FB_ERR_INVALID_ARG),
            (lambda: fb.Rope([math.nan]), fb.FB_ERR_INVALID_ARG)):
        with pytest.raises(fb.FlashBiasError) as e:
            call()
        assert e.value.status == status
    torch.cuda.synchronize()
    assert _status() == fb.FB_OK


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("context", [0, 70, 9000])
def test_non_finite_values_in_two_row_tiles(kind, context):
    """150 rows, so two row tiles, whose keys one CTA or many have: a non-finite value of a new token reaches the rows
    that see it, in its channel, and nothing else, to the bit."""
    T, hot = 150, 100
    c = _case(kind, 64, 2, 2, T, 16, [context, 33], None, "low8", False, seed=11)
    clean = _call(c)
    at = int(c["table"][0, (context + hot) // 16]), 1, (context + hot) % 16, 5
    if kind == "bf16":
        c["cache"].v[at] = -math.inf
    else:
        c["cache"].v.view(torch.uint8)[at] = 0x7F
    o, lse = _call(c)
    assert torch.equal(lse, clean[1])
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[0, 1, hot:, 5] = True
    assert torch.equal(o[~hit], clean[0][~hit])
    assert (o[hit] == -math.inf).all() if kind == "bf16" else o[hit].isnan().all()
    assert _status() == fb.FB_OK


@pytest.mark.parametrize("kind,d,Hq,H,T,page,prefix,counts,bias,tree", [
    ("bf16", 128, 16, 1, 17, 16, [40000], None, "none", False),  # one item over all CTAs, two row tiles
    ("e4m3", 128, 4, 1, 70, 64, [0, 1, 95, 96, 97], [70, 1, 0, 70, 69], "low64", True),
    ("e4m3", 128, 8, 2, 40, 16, [700, 20000], None, "low100", True),  # one row tile, one slot of keys
    ("bf16", 64, 2, 1, 300, 32, [1234], None, "sandwich128", False),
    ("e4m3", 32, 40, 2, 20, 256, [5000] * 3, [20, 0, 7], "alibi", True),  # chunks of 256 rows
    ("bf16", 96, 1, 1, 24, 16, [30000], None, "alibi", True),  # one split row tile over all CTAs
])
def test_tiles_at_their_borders(kind, d, Hq, H, T, page, prefix, counts, bias, tree):
    c = _case(kind, d, Hq, H, T, page, prefix, counts, bias, tree, seed=21)
    ws = fb.cache_workspace(len(prefix), Hq, H, T, d)
    want, got = _want(c), _call(c, workspace=ws)
    assert _status() == fb.FB_OK
    _compare(got, want)
    for _ in range(3):
        again = _call(c, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_two_streams_with_workspaces_of_their_own():
    """Calls that overlap: the same cache read by two streams at once gives each what it gets alone."""
    cases = [_case("e4m3", 128, 8, 2, T, 64, [6000, 900], None, "none", False, seed=30 + T) for T in (1, 40)]
    alone = [_call(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    spaces = [fb.cache_workspace(2, 8, 2, c["q"].shape[2], 128) for c in cases]
    torch.cuda.synchronize()
    for _ in range(4):
        out = []
        for c, s, w in zip(cases, streams, spaces):
            with torch.cuda.stream(s):
                out.append(_call(c, workspace=w))
        torch.cuda.synchronize()
        for a, b in zip(out, alone):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert _status() == fb.FB_OK


def _plant(c, kind, b, head, token, channel, what=math.inf):
    """`what` (NaN in an 8-bit cache) at one value of cache token `token` of sequence b."""
    page = c["cache"].page
    at = int(c["table"][b, token // page]), head, token % page, channel
    if kind == "bf16":
        c["cache"].v[at] = what
    else:
        c["cache"].v.view(torch.uint8)[at] = 0x7F


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("bias", ["none", "alibi", "low8"])
def test_non_finite_values_in_many_short_items(kind, bias):
    """Many items whose keys one CTA has, one after the other: a non-finite value of a new token, in every third
    sequence, reaches all rows that see it and nothing of the next item."""
    B, H, T, d = 160, 16, 4, 32
    c = _case(kind, d, H, H, T, 16, [(7 * b) % 40 for b in range(B)], None, bias, True, seed=41)
    clean = _call(c)
    hit = torch.zeros(B, H, T, d, dtype=torch.bool)
    for b in range(0, B, 3):
        h, u = b % H, b % T
        _plant(c, kind, b, h, int(c["prefix"][b]) + u, 9)
        hit[b, h, :, 9] = ((c["mask"][b, :, 0] >> u) & 1).bool()
    hit = hit.cuda()
    ws = fb.cache_workspace(B, H, H, T, d)
    for _ in range(5):
        o, lse = _call(c, workspace=ws)
        assert torch.equal(lse, clean[1]) and torch.equal(o[~hit], clean[0][~hit])
        assert (o[hit] == math.inf).all() if kind == "bf16" else o[hit].isnan().all()
    assert _status() == fb.FB_OK


@pytest.mark.parametrize("B,H,T,context", [(20, 8, 300, 0), (12, 6, 260, 90), (50, 3, 140, 5)])
def test_many_short_items_of_two_row_tiles(B, H, T, context):
    """Items of one to four key tiles, most of which one CTA has, between items that cross CTAs: chunks of both row
    tiles and of one in turn."""
    c = _case("bf16", 32, H, H, T, 16, [context + b % 7 for b in range(B)], None, "none", False, seed=61)
    ws = fb.cache_workspace(B, H, H, T, 32)
    got = _call(c, workspace=ws)
    _compare(got, _want(c))
    for _ in range(5):
        again = _call(c, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert _status() == fb.FB_OK


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("T", [99, 100, 128])
@pytest.mark.parametrize("context", [0, 200, 9000])
@pytest.mark.parametrize("late", [False, True])
def test_non_finite_values_in_a_split_row_tile(kind, T, context, late):
    """One row tile, whose key tiles two streams take in turn, and one CTA or many. A row may see nothing but its own key,
    which the second stream has, or keys of the first whose weight is nothing beside those of the second: the value
    reaches the rows that see it, in its channel, as it is."""
    c = _case(kind, 64, 2, 2, T, 16, [context, 3], None, "none", False, seed=43)
    see = torch.ones(T, T, dtype=torch.bool).tril()
    if late:
        P = context + T + 16
        fk = torch.zeros(1, P, 1)
        fk[0, context + 96:] = 200.0  # e^200 times the weight of the keys before
        c["fq"], c["fk"] = torch.ones(1, P, 1), fk
    else:
        see[T - 3:] = torch.eye(T, dtype=torch.bool)[T - 3:]
    c["mask"] = _words(see[None].expand(2, T, T))
    clean = _call(c)
    hit = torch.zeros_like(clean[0], dtype=torch.bool)
    for u, channel in ((T - 3, 5), (T - 1, 63)):
        _plant(c, kind, 0, 1, context + u, channel)
        hit[0, 1, see[:, u].nonzero()[:, 0].cuda(), channel] = True
    o, lse = _call(c)
    assert torch.equal(lse, clean[1]) and torch.equal(o[~hit], clean[0][~hit])
    assert (o[hit] == math.inf).all() if kind == "bf16" else o[hit].isnan().all()
    assert _status() == fb.FB_OK


@pytest.mark.parametrize("T,context", [(24, 0), (24, 500), (100, 10), (150, 90)])
def test_values_beyond_bf16_in_the_tiles(T, context):
    """A finite value that its code and scale carry past bf16's range (3.4e38 is written as 2^128) is infinite in the
    128-row tiles, for a new token as for one of the context: the rows that see it get it, the others nothing."""
    c = _case("e4m3", 64, 2, 2, T, 16, [context, 3], None, "none", False, seed=45)
    clean = _call(c)
    hot = T - 2
    row = torch.zeros(2, 2, 1, 64)
    row[:, :, 0, 11], row[:, :, 0, 12] = 3.4e38, -3.4e38
    at = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pool, scale = c["cache"].k.clone(), c["cache"].k_scale.clone()
    fb.cache_write(c["cache"], row.cuda(), row.cuda(), c["table"].cuda(), at([context + hot, 3 + hot]), at([1, 0]))
    c["cache"].k.copy_(pool)
    c["cache"].k_scale.copy_(scale)
    o, lse = _call(c)
    assert torch.equal(lse, clean[1])
    assert (o[0, :, hot:, 11] == math.inf).all() and (o[0, :, hot:, 12] == -math.inf).all()
    assert torch.equal(o[0, :, :hot], clean[0][0, :, :hot]) and torch.equal(o[1], clean[0][1])
    assert torch.isfinite(o[0, :, hot:, :11]).all() and torch.isfinite(o[0, :, hot:, 13:]).all()
    assert _status() == fb.FB_OK


@pytest.mark.parametrize("d", [16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("T", [1, 5, 24])
@pytest.mark.parametrize("channel", [0, 3, 7, 12])
def test_infinite_keys(d, T, channel):
    """A key whose score is -inf has no weight, whatever the head dim: the result is, to the bit, that of a key whose
    score is so low that its weight is 0."""
    c = _case("bf16", d, 2, 2, T, 16, [40], None, "none", False, seed=47)
    c["q"][..., channel] = c["q"][..., channel].abs() + 0.5
    at = int(c["table"][0, 1]), slice(None), 5, channel  # context token 21
    c["cache"].k[at] = -1e38
    low = _call(c)
    c["cache"].k[at] = -math.inf
    got = _call(c)
    assert torch.isfinite(low[0]).all()
    assert torch.equal(got[0], low[0]) and torch.equal(got[1], low[1])
    assert _status() == fb.FB_OK


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("T", [1, 16, 17, 40, 150])
@pytest.mark.parametrize("R", [3, 8, 40])
def test_nan_factors_reach_their_rows(kind, T, R):
    """A NaN in a query position's factors makes the rows of that position NaN, whatever kernel their number takes; the
    other rows keep their results."""
    c = _case(kind, 64, 2, 2, T, 16, [50], None, f"low{R}", False, seed=49)
    c["fq"][0, 0, R - 1] = 2 * c["fq"].abs().max()  # the column's size stays when another value becomes NaN
    clean = _call(c)
    assert _status() == fb.FB_OK
    c["fq"][1, 50 + T - 1, R - 1] = math.nan
    o, lse = _call(c)
    assert _status() == (fb.FB_OK if R <= 4 else fb.FB_ERR_RANGE)
    hit = torch.zeros(1, 2, T, dtype=torch.bool, device="cuda")
    hit[0, 1, T - 1] = True
    assert o[hit].isnan().all() and lse[hit].isnan().all()
    assert torch.equal(o[~hit], clean[0][~hit]) and torch.equal(lse[~hit], clean[1][~hit])


def test_reserved_and_least_scale_bytes_read_back():
    """Byte 255 is NaN and byte 0 is 2^-127, as the type of the scales says."""
    cache = _cache(1, 2, 16, 32, "e4m3", 51)
    cache.k_scale.view(torch.uint8)[0, :, 3] = 255
    cache.v_scale.view(torch.uint8)[0, :, 4] = 0
    cache.v_scale.view(torch.uint8)[0, :, 5] = 255
    cache.v.view(torch.uint8)[0, :, 5] = 0
    tab = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        k, v = fb.cache_read(cache, tab, None, None, 16, dtype=dtype)
        assert k[0, :, 3].isnan().all() and v[0, :, 5].isnan().all()
        least = ref.e4m3_values(cache.v.view(torch.uint8)[0, :, 4].cpu()) * 2.0 ** -127
        assert torch.equal(v[0, :, 4].cpu().to(F64), least.to(dtype).to(F64))
        assert torch.isfinite(k[0, :, [i for i in range(16) if i != 3]]).all()
        assert torch.isfinite(v[0, :, [i for i in range(16) if i != 5]]).all()
    assert _status() == fb.FB_OK


@pytest.mark.parametrize("T", [1, 6, 24])
def test_least_scales_of_keys(T):
    """Keys with the scale 2^-127 against queries near the largest: ordinary scores, in both kernels."""
    c = _case("e4m3", 64, 2, 2, T, 16, [60], None, "none", False, seed=53)
    c["q"] = (c["q"].float() * 2.0 ** 121).to(torch.bfloat16)
    c["cache"].k_scale.view(torch.uint8).zero_()
    o, lse, to, tl = _want(c)
    assert float(lse.max()) - math.log(61) > 0.05  # the scores matter
    # the tiles hold keys as bf16, whose step below 2^-126 is 2^-133: half of it for each value of a key
    off = 2.0 ** -134 * c["q"].to(F64).abs().sum(-1) / 8 if T > 16 else torch.zeros(1, 2, T, dtype=F64)
    weight = ref.rows(ref.pool_values(c["cache"].v.cpu(), c["cache"].v_scale.cpu()), c["table"][0], 0, 60 + T).abs().amax()
    _compare(_call(c), (o, lse, to + 2 * off[..., None] * weight, tl + off))


@pytest.mark.parametrize("T", [1, 6, 24])
def test_scale_byte_of_nan(T):
    """A key row whose scale is NaN makes the rows that see it NaN."""
    c = _case("e4m3", 64, 2, 2, T, 16, [20], None, "none", False, seed=55)
    clean = _call(c)
    c["cache"].k_scale.view(torch.uint8)[int(c["table"][0, (20 + T - 1) // 16]), 1, (20 + T - 1) % 16] = 255
    o, lse = _call(c)
    hit = torch.zeros(1, 2, T, dtype=torch.bool, device="cuda")
    hit[0, 1, T - 1] = True
    assert o[hit].isnan().all() and lse[hit].isnan().all()
    assert torch.equal(o[~hit], clean[0][~hit]) and torch.equal(lse[~hit], clean[1][~hit])
    assert _status() == fb.FB_OK


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("T", [1, 3, 24])
def test_values_beside_a_page_that_is_not_there(kind, T):
    """A page of the context that the table does not lead to is not seen; a non-finite value in the page beside it, which
    every row sees, stays."""
    c = _case(kind, 64, 2, 2, T, 16, [60], None, "none", False, seed=57)
    c["table"][0, 1] = -1
    clean = _call(c)
    assert _status() == fb.FB_ERR_RANGE and torch.isfinite(clean[0]).all()
    _plant(c, kind, 0, 1, 3, 7)
    o, lse = _call(c)
    assert _status() == fb.FB_ERR_RANGE
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[0, 1, :, 7] = True
    assert torch.equal(lse, clean[1]) and torch.equal(o[~hit], clean[0][~hit])
    assert (o[hit] == math.inf).all() if kind == "bf16" else o[hit].isnan().all()


@pytest.mark.parametrize("T", [1, 24])
@pytest.mark.parametrize("side", ["fq", "fk"])
def test_factor_columns_of_zeros(T, side):
    """A column that is zero on one side adds nothing, however large the other side is, and is no error."""
    c = _case("bf16", 64, 2, 2, T, 16, [40], None, "low8", False, seed=59)
    other = "fk" if side == "fq" else "fq"
    c[side][..., 2] = 0.0
    want = _want(c)
    c[other][..., 2] = _randn(c[other].shape[:2], 60) * 1e9
    got = _call(c)
    assert _status() == fb.FB_OK
    _compare(got, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("first", [0, 123456, 2 ** 24])
def test_rope_of_pairs_of_very_different_size(dtype, inter, first):
    """Each pair is turned to its own size: the bound is of its two values (angle, sine, cosine and products within
    2^-21 of them, one rounding), not of the head's largest."""
    B, H, N, d, rot = 1, 3, 130, 64, 48
    r = fb.Rope.scaled(rot, interleaved=inter, factor=1.5)
    p = torch.arange(rot // 2)
    ia, ib = (2 * p, 2 * p + 1) if inter else (p, p + rot // 2)
    size = torch.ones(d)
    size[ia] = size[ib] = torch.exp2(-40.0 * p / p[-1])
    x = (_randn((B, H, N, d), 63) * size).to(dtype)
    pos = (torch.arange(N) + first).to(torch.int32)
    for call, sign in ((fb.rope, 1.0), (fb.rope_bwd, -1.0)):
        y, _ = call(x.cuda(), None, r, pos.cuda())
        want = ref.rope(x, r.frequencies, pos[None], rot, inter, r.factor, sign)
        big = torch.zeros_like(want)
        big[..., ia] = big[..., ib] = torch.maximum(x[..., ia].abs(), x[..., ib].abs()).to(F64) * r.factor
        err = (y.cpu().to(F64) - want).abs()
        assert (err <= torch.finfo(dtype).eps / 2 * want.abs() + 2.0 ** -21 * 2 * big).all()
    assert _status() == fb.FB_OK


@pytest.mark.parametrize("T", [3, 24, 150])
@pytest.mark.parametrize("by", ["key", "bias"])
def test_non_finite_values_of_keys_without_weight(T, by):
    """Infinite values of a context token and a new one whose score is -inf, or shut out by the bias: what 0 times
    infinity makes of their channels is open, the other channels and the rows that do not see them keep their results."""
    c = _case("bf16", 64, 1, 1, T, 16, [40], None, "none", False, seed=65)
    page = lambda i: (int(c["table"][0, i // 16]), 0, i % 16)  # noqa: E731
    if by == "key":
        c["q"][..., 2] = c["q"][..., 2].abs() + 0.5
        for i in (7, 41):
            c["cache"].k[page(i) + (2,)] = -math.inf
    else:
        fk = torch.zeros(1, 48 + T, 1)
        fk[0, 7] = fk[0, 41] = 1.0
        c["fq"], c["fk"] = torch.full((1, 48 + T, 1), -1e38), fk
    clean = _call(c)
    c["cache"].v[page(7) + (10,)] = math.inf
    c["cache"].v[page(41) + (20,)] = -math.inf
    o, lse = _call(c)
    open_ = torch.zeros_like(o, dtype=torch.bool)
    open_[..., 10] = True
    open_[0, 0, 1:, 20] = True
    assert torch.isfinite(clean[0]).all() and torch.equal(lse, clean[1]) and torch.equal(o[~open_], clean[0][~open_])
    assert _status() == fb.FB_OK
