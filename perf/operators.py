"""The cases by which the serving operators are measured: rotary positions (with
their gradient), the paged key/value cache that is written and read back, and
the attention of new tokens, a single one or a drafted tree, over that cache
with a low-rank additive bias.

Each case goes through the operators twice: in plain form, elementary torch
operations in 32 bits, and (`own` true) through the calls that a user makes of
the package. `exact` is the same result in 64 bits from the definition.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3_MAX = 448.0


# --------------------------------------------------------------------- cases

def listed():
    return [
        # one new token of each of 8 sequences of the 12-head, head-dim-64 language model: the call every decode step makes
        dict(name="rope_token", op="rope", batch=8, q_heads=12, kv_heads=12, tokens=1, dim=64, rotary=64,
             interleaved=False, scaling="none", first=2047, type="bf16", layout="bnhd"),
        # the same model's prompt of 2048 tokens, queries and keys as the projection leaves them (token-major)
        dict(name="rope_prompt", op="rope", batch=8, q_heads=12, kv_heads=12, tokens=2048, dim=64, rotary=64,
             interleaved=False, scaling="none", first=0, type="bf16", layout="bnhd"),
        # training on long documents with grouped heads: the gradient at far positions, half of each head rotated
        dict(name="rope_far_grad", op="rope_grad", batch=1, q_heads=32, kv_heads=8, tokens=16384, dim=128, rotary=64,
             interleaved=True, scaling="yarn", first=100000, type="bf16", layout="bhnd"),
        # a decode step's keys and values of 64 sequences go into an 8-bit cache
        dict(name="write_token", op="write", batch=64, kv_heads=8, tokens=1, dim=128, page=64, cache="e4m3",
             type="bf16", start=500, layout="bnhd"),
        # 8 ragged prompts of the 12-head model fill an 8-bit cache of small pages
        dict(name="write_prompt", op="write", batch=8, kv_heads=12, tokens=2048, dim=64, page=16, cache="e4m3",
             type="bf16", start=0, layout="bhnd"),
        # a few odd lengths read back from a 16-bit cache
        dict(name="read_short", op="read", batch=3, kv_heads=4, tokens=777, dim=80, page=32, cache="bf16", type="bf16",
             start=5),
        # four long contexts read back from the 8-bit cache, for a pass of full attention over them
        dict(name="read_long", op="read", batch=4, kv_heads=8, tokens=32768, dim=128, page=64, cache="e4m3",
             type="bf16", start=0),
        # a single user's next token with Sandwich factors: latency
        dict(name="token_short", op="attend", batch=1, q_heads=12, kv_heads=12, context=700, tokens=1, dim=64, page=16,
             cache="bf16", bias="sandwich", rank=64, tree=False),
        # a decode step of the 16-head ALiBi model, ragged contexts up to 8192, 8-bit cache
        dict(name="token_alibi", op="attend", batch=16, q_heads=16, kv_heads=16, context=8191, tokens=1, dim=128,
             page=64, cache="e4m3", bias="alibi", rank=2, tree=False),
        # two very long contexts with grouped heads and no bias (rotary positions), 16-bit cache
        dict(name="token_long", op="attend", batch=2, q_heads=32, kv_heads=8, context=131071, tokens=1, dim=128,
             page=128, cache="bf16", bias="none", rank=0, tree=False),
        # trees of 24 drafted tokens checked by the 12-head Sandwich model
        dict(name="tree", op="attend", batch=8, q_heads=12, kv_heads=12, context=2024, tokens=24, dim=64, page=16,
             cache="bf16", bias="sandwich", rank=64, tree=True),
        # trees of 61 drafted tokens, grouped heads, per-head factors of rank 32, 8-bit cache
        dict(name="tree_grouped", op="attend", batch=16, q_heads=32, kv_heads=8, context=8131, tokens=61, dim=128,
             page=64, cache="e4m3", bias="lowrank", rank=32, tree=True),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rope", "rope_grad", "write", "read", "attend", "attend", "attend"])
    group = rng.choice([1, 1, 2, 4, 8])
    kv = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
    dim = rng.choice([32, 48, 64, 64, 80, 96, 128, 128])
    if op in ("rope", "rope_grad"):
        group = min(group, max(1, 32 // kv))
        tokens, batch = log(1, 16384), log(1, 64)
        most = 40 * 16384 * 128
        batch = max(1, min(batch, most // ((group + 1) * kv * tokens * dim)))
        tokens = max(1, min(tokens, most // ((group + 1) * kv * batch * dim)))
        kind = rng.choice(["bf16", "bf16", "f32"])
        if kind == "f32":
            tokens = max(1, tokens // 2)
        rotary = rng.choice([dim, dim, dim // 2, dim // 4])
        return dict(op=op, batch=batch, q_heads=kv * group, kv_heads=kv, tokens=tokens, dim=dim, rotary=rotary,
                    interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "yarn"]),
                    first=log(1, 1000000) - 1, type=kind, layout=rng.choice(["bhnd", "bnhd"]))
    page = rng.choice([16, 32, 64, 128])
    cache = rng.choice(["bf16", "e4m3"])
    if op in ("write", "read"):
        tokens, batch = log(1, 32768 if op == "read" else 4096), log(1, 64)
        most = 4 * 8 * 32768 * 128 if op == "read" else 8 * 12 * 2048 * 64
        batch = max(1, min(batch, most // (kv * tokens * dim)))
        tokens = max(1, min(tokens, most // (kv * batch * dim)))
        c = dict(op=op, batch=batch, kv_heads=kv, tokens=tokens, dim=dim, page=page, cache=cache,
                 type=rng.choice(["bf16", "bf16", "f32"]), start=log(1, 700) - 1)
        if c["type"] == "f32":
            c["batch"] = max(1, batch // 2)
            c["tokens"] = max(1, tokens // 2)
        if op == "write":
            c["layout"] = rng.choice(["bhnd", "bnhd"])
        return c
    tree = rng.random() < 0.6
    tokens = log(1, 64) if tree else 1
    batch, context = log(1, 32), log(1, 65536)
    group = min(group, max(1, 32 // kv))
    most_bytes, most_pairs = 900e6, 16 * 32 * 61 * 3300
    size = 2 * kv * dim * (2 if cache == "bf16" else 1)
    context = max(1, min(context, int(most_bytes / (size * batch)), int(most_pairs / (batch * kv * group * tokens))))
    bias = rng.choice(["none", "alibi", "sandwich", "lowrank"])
    rank = {"none": 0, "alibi": 2, "sandwich": rng.choice([32, 64, 128]), "lowrank": rng.choice([3, 8, 17, 32, 48])}[bias]
    return dict(op=op, batch=batch, q_heads=kv * group, kv_heads=kv, context=context, tokens=tokens, dim=dim, page=page,
                cache=cache, bias=bias, rank=rank, tree=tree)


# ------------------------------------------------------- what a case is made of

def lengths(case):
    """Context of each sequence before its new tokens: ragged, the longest first."""
    n, batch = case["context"], case["batch"]
    return [n - (b * 7919) % (n // 2 + 1) if b else n for b in range(batch)]


def new_counts(case):
    """New tokens of each sequence: the last of a batch of trees bring fewer."""
    t = case["tokens"]
    return [t - (b * 5) % (t // 2 + 1) if case.get("tree") else t for b in range(case["batch"])]


def row_counts(case):
    """Tokens of each sequence that are written or read: ragged, the longest first."""
    t = case["tokens"]
    return [t - (b * 6007) % (t // 2 + 1) if b else t for b in range(case["batch"])]


def frequencies(case):
    """Angle per position of each rotated pair, and the factor on the result."""
    rot, base = case["rotary"], 10000.0
    w = [base ** (-2.0 * k / rot) for k in range(rot // 2)]
    if case["scaling"] == "linear":
        return [x / 4.0 for x in w], 1.0
    if case["scaling"] == "yarn":  # 16 times the length of training (4096): slow pairs are stretched, fast ones stay
        s, trained, fast, slow = 16.0, 4096.0, 32.0, 1.0

        def turn(n):
            return rot * math.log(trained / (n * 2 * math.pi)) / (2 * math.log(base))

        lo, hi = max(math.floor(turn(fast)), 0), min(math.ceil(turn(slow)), rot - 1)
        keep = [1.0 - min(max((k - lo) / max(hi - lo, 0.001), 0.0), 1.0) for k in range(rot // 2)]
        return [x / s * (1 - a) + x * a for x, a in zip(w, keep)], 0.1 * math.log(s) + 1.0
    return w, 1.0


def tree_of(tokens, rng):
    """A drafted tree: each token's parent is an earlier one, or the context (-1)."""
    parents = [-1]
    for t in range(1, tokens):
        parents.append(rng.randint(max(-1, t - 6), t - 1))
    return parents


def normal(shape, gen, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def quantised(x):
    """8-bit values and the exponents of their power-of-two scales, one for each row of x:
    the least scale (2^-126 or more) under which no value passes 448."""
    x = x.float()
    top = x.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(top)  # top = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = (e - 9 + (m > 0.875).int()).clamp(min=-126)
    e = torch.where(top > 0, e, torch.full_like(e, -126))
    codes = (x * ((127 - e) << 23).view(torch.float32)).to(torch.float8_e4m3fn)  # 2^-e, from its bits
    return codes, (e + 127).to(torch.uint8).squeeze(-1).view(torch.float8_e8m0fnu)


def unquantised(codes, scale):
    """The values that 8-bit codes and their scales stand for, in 32 bits."""
    return codes.float() * scale.float().unsqueeze(-1)


def prepare(case, seed):
    import random
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    B, d, s = case["batch"], case["dim"], {"case": case}

    def heads(h, n, dtype):  # [B, h, n, d], in the memory order of the case's layout
        if case.get("layout") == "bnhd":
            return normal((B, n, h, d), gen, dtype).transpose(1, 2)
        return normal((B, h, n, d), gen, dtype)

    if case["op"] in ("rope", "rope_grad"):
        dt, n = TYPES[case["type"]], case["tokens"]
        s["q"], s["k"] = heads(case["q_heads"], n, dt), heads(case["kv_heads"], n, dt)
        first = torch.tensor([case["first"] + rng.randint(0, 50) for _ in range(B)], dtype=torch.int32, device="cuda")
        s["positions"] = first[:, None] + torch.arange(n, dtype=torch.int32, device="cuda")
        w, s["factor"] = frequencies(case)
        s["freq"] = torch.tensor(w, dtype=torch.float64, device="cuda")
        if own:
            import attention_rank_additive_b200 as fb
            s["rope"] = fb.Rope(w, interleaved=case["interleaved"], factor=s["factor"])
        return s

    H, page = case["kv_heads"], case["page"]
    if case["op"] == "attend":
        last = [a + b for a, b in zip(lengths(case), [case["tokens"]] * B)]
    else:
        s["starts"] = [case["start"] + rng.randint(0, 9) for _ in range(B)]
        last = [x + case["tokens"] for x in s["starts"]]
    per = max(-(-n // page) for n in last)
    total = B * per + 3
    order = torch.randperm(total, generator=gen, device="cuda")[: B * per].to(torch.int32)
    s["table"] = order.view(B, per).contiguous()
    kv = [normal((total, H, page, d), gen, torch.bfloat16) for _ in range(2)]
    if case["cache"] == "e4m3":
        s["k"], s["k_scale"] = quantised(kv[0])
        s["v"], s["v_scale"] = quantised(kv[1])
    else:
        s["k"], s["v"], s["k_scale"], s["v_scale"] = kv[0], kv[1], None, None

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    if case["op"] in ("write", "read"):
        s["starts"], s["counts"] = ints(s["starts"]), ints(row_counts(case))
        if case["op"] == "write":
            dt = TYPES[case["type"]]
            s["new_k"], s["new_v"] = heads(H, case["tokens"], dt), heads(H, case["tokens"], dt)
    else:
        T, Hq, R = case["tokens"], case["q_heads"], case["rank"]
        s["q"] = normal((B, Hq, T, d), gen, torch.bfloat16)
        s["prefix"], s["counts"] = ints(lengths(case)), ints(new_counts(case))
        s["mask"] = s["depth"] = None
        if case["tree"]:
            seen, depth = torch.zeros((B, T, T), dtype=torch.bool), torch.zeros((B, T), dtype=torch.int32)
            for b in range(B):
                for t, p in enumerate(tree_of(T, rng)):
                    if p >= 0:
                        seen[b, t] = seen[b, p]
                        depth[b, t] = depth[b, p] + 1
                    seen[b, t, t] = True
            bits = torch.zeros((B, T, -(-T // 32) * 32), dtype=torch.int64)
            bits[:, :, :T] = seen
            words = (bits.view(B, T, -1, 32) << torch.arange(32)).sum(-1)
            s["mask"] = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32).cuda()  # [B, T, words]
            s["depth"] = depth.cuda()
        P = max(last)
        s["phi_q"] = s["phi_k"] = None
        pos = torch.arange(P, device="cuda", dtype=torch.float64)
        if case["bias"] == "sandwich":
            w = 10000.0 ** (-2.0 * torch.arange(1, R // 2 + 1, device="cuda", dtype=torch.float64) / R)
            a = pos[:, None] * w
            s["phi_q"] = s["phi_k"] = torch.stack([a.cos(), a.sin()], -1).reshape(1, P, R).float()
        elif case["bias"] == "alibi":  # -m_h (i - j), the slope on the query's side so that grouped heads share a key's
            m = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, device="cuda", dtype=torch.float64) / Hq)
            s["phi_q"] = torch.stack([-m[:, None] * pos, m[:, None].expand(Hq, P)], -1).float().contiguous()
            s["phi_k"] = torch.stack([torch.ones_like(pos), pos], -1).float().view(1, P, 2)
        elif case["bias"] == "lowrank":
            s["phi_q"] = normal((Hq, P, R), gen, torch.float32) * R ** -0.5
            s["phi_k"] = normal((H, P, R), gen, torch.float32)
        if own:
            import attention_rank_additive_b200 as fb
            s["bias"] = fb.CacheBias(s["phi_q"], s["phi_k"]) if R else None
            s["workspace"] = fb.cache_workspace(B, Hq, H, T, d)
    if own:
        import attention_rank_additive_b200 as fb
        s["cache"] = fb.PagedCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    return s


# ---------------------------------------------------------------- the passes

def rotated(x, angle, case, factor, sign):
    """x with its first `rotary` values turned by sign * angle ([B, 1, N, pairs], 64 bits) and multiplied by factor."""
    rot = case["rotary"]
    c, s = (angle.cos() * factor).float(), (angle.sin() * (factor * sign)).float()
    y = x.float()
    if case["interleaved"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    else:
        a, b = y[..., : rot // 2], y[..., rot // 2: rot]
        turned = torch.cat([a * c - b * s, a * s + b * c], -1)
    return torch.cat([turned, y[..., rot:]], -1).to(x.dtype)


def places(table, index, page):
    """(page, place in it) of the tokens at `index` [B, n] of each sequence."""
    return table.long().gather(1, index // page), index % page


def plain_rope(s):
    case = s["case"]
    angle = (s["positions"].double()[:, None, :, None]) * s["freq"]
    sign = -1.0 if case["op"] == "rope_grad" else 1.0
    return [rotated(s[x], angle, case, s["factor"], sign) for x in ("q", "k")]


def plain_write(s):
    case = s["case"]
    t = torch.arange(case["tokens"], device="cuda")
    at, place = places(s["table"], s["starts"].long()[:, None] + t, case["page"])
    real = (t < s["counts"][:, None])[..., None]  # [B, n, 1]
    for new, name in ((s["new_k"], "k"), (s["new_v"], "v")):
        pool, new = s[name], new.transpose(1, 2)  # [B, n, H, d]
        if case["cache"] == "e4m3":
            codes, scale = quantised(new)
            scales = s[name + "_scale"].view(torch.uint8)
            scales[at, :, place] = torch.where(real, scale.view(torch.uint8), scales[at, :, place])
            pool, new = pool.view(torch.uint8), codes.view(torch.uint8)
        pool[at, :, place] = torch.where(real[..., None], new.to(pool.dtype), pool[at, :, place])
    return [x for x in (s["k"], s["v"], s["k_scale"], s["v_scale"]) if x is not None]


def gathered(s, name, at, place):
    """Rows of the cache at (at, place) [B, n], in 32 bits: [B, H, n, d]."""
    if s["case"]["cache"] == "e4m3":
        codes = s[name].view(torch.uint8)[at, :, place].view(torch.float8_e4m3fn)
        x = unquantised(codes, s[name + "_scale"].view(torch.uint8)[at, :, place].view(torch.float8_e8m0fnu))
    else:
        x = s[name][at, :, place].float()
    return x.transpose(1, 2)


def plain_read(s):
    case = s["case"]
    t = torch.arange(case["tokens"], device="cuda")
    at, place = places(s["table"], s["starts"].long()[:, None] + t, case["page"])
    real = (t < s["counts"][:, None])[:, None, :, None]
    return [torch.where(real, gathered(s, x, at, place), 0.0).to(TYPES[case["type"]]).contiguous() for x in ("k", "v")]


def plain_attend(s):
    case = s["case"]
    B, Hq, H, T, d = case["batch"], case["q_heads"], case["kv_heads"], case["tokens"], case["dim"]
    G, N = Hq // H, case["context"] + T
    prefix, counts = s["prefix"].long(), s["counts"].long()
    j, t = torch.arange(N, device="cuda"), torch.arange(T, device="cuda")
    last = s["table"].shape[1] * case["page"] - 1
    at, place = places(s["table"], j.clamp(max=last).expand(B, N), case["page"])
    u = (j - prefix[:, None])  # a key's number among the new tokens; negative in the context
    new = u.clamp(0, T - 1)
    if case["tree"]:
        word = s["mask"].long().gather(2, (new // 32)[:, None].expand(B, T, N))
        seen = (word >> (new % 32)[:, None]) & 1 > 0
        depth = s["depth"].long()
    else:
        seen, depth = new[:, None] <= t[:, None], t.expand(B, T)
    real = counts[:, None, None]
    seen = torch.where(u[:, None] < 0, torch.ones_like(seen), seen & (u[:, None] < real)) & (t[:, None] < real)
    seen = seen[:, None, None]  # [B, 1, 1, T, N]
    k, v = gathered(s, "k", at, place), gathered(s, "v", at, place)
    q = s["q"].float().view(B, H, G * T, d)
    x = (torch.matmul(q, k.transpose(2, 3)) * d ** -0.5).view(B, H, G, T, N)
    if case["rank"]:
        P = s["phi_q"].shape[1]
        qpos = (prefix[:, None] + depth).clamp(max=P - 1)
        kpos = torch.where(u < 0, j, prefix[:, None] + depth.gather(1, new)).clamp(max=P - 1)
        fq, fk = s["phi_q"][:, qpos].transpose(0, 1), s["phi_k"][:, kpos].transpose(0, 1)  # [B, heads, n, R]
        fq = fq.expand(B, Hq, T, -1).reshape(B, H, G * T, -1)
        x = x + torch.matmul(fq, fk.expand(B, H, N, -1).transpose(2, 3)).view(B, H, G, T, N)
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, H, G * T, N), v).view(B, H, G, T, d)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + torch.log(total)).view(B, Hq, T)
    return [o.to(torch.bfloat16).view(B, Hq, T, d), lse]


def own_run(s):
    import attention_rank_additive_b200 as fb
    op = s["case"]["op"]
    if op == "rope":
        return fb.rope(s["q"], s["k"], s["rope"], s["positions"])
    if op == "rope_grad":
        return fb.rope_bwd(s["q"], s["k"], s["rope"], s["positions"])
    if op == "write":
        fb.cache_write(s["cache"], s["new_k"], s["new_v"], s["table"], s["starts"], s["counts"])
        return [x for x in (s["k"], s["v"], s["k_scale"], s["v_scale"]) if x is not None]
    if op == "read":
        return fb.cache_read(s["cache"], s["table"], s["starts"], s["counts"], s["case"]["tokens"],
                             dtype=TYPES[s["case"]["type"]])
    return fb.attn_cache(s["q"], s["cache"], s["table"], s["prefix"], s["counts"], tree_mask=s["mask"],
                         depths=s["depth"], bias=s["bias"], workspace=s["workspace"])


def run(state):
    if own:
        return own_run(state)
    op = state["case"]["op"]
    if op in ("rope", "rope_grad"):
        return plain_rope(state)
    return {"write": plain_write, "read": plain_read, "attend": plain_attend}[op](state)


# ------------------------------------------------------------- work and truth

def work(case):
    B, d = case["batch"], case["dim"]
    if case["op"] in ("rope", "rope_grad"):
        size = 2 if case["type"] == "bf16" else 4
        values = B * (case["q_heads"] + case["kv_heads"]) * case["tokens"]
        return {"bytes": values * d * size * 2 + B * case["tokens"] * 4 + case["rotary"] * 4,
                "flops": values * case["rotary"] * 3}
    H, held = case["kv_heads"], (d + 1 if case["cache"] == "e4m3" else 2 * d)
    if case["op"] in ("write", "read"):
        size = 2 if case["type"] == "bf16" else 4
        rows = 2 * H * sum(row_counts(case))
        outside = rows if case["op"] == "write" else 2 * H * B * case["tokens"]
        tables = 8 * B + 4 * sum(-(-n // case["page"]) for n in row_counts(case))
        return {"bytes": rows * held + outside * d * size + tables, "flops": 2 * rows * d}
    pre, new = lengths(case), new_counts(case)
    Hq, T, R, G = case["q_heads"], case["tokens"], case["rank"], case["q_heads"] // H
    keys = sum(a + b for a, b in zip(pre, new))
    pairs = sum((a + (1 + min(b, 6)) / 2) * b if case["tree"] else a + 1 for a, b in zip(pre, new)) * Hq
    tables = 4 * sum(-(-(a + b) // case["page"]) for a, b in zip(pre, new)) + 8 * B
    factors = 0
    if R:
        rows_k = (max(pre) + T) * R * 4 * (H if case["bias"] == "lowrank" else 1)
        rows_q = sum(new) * R * 4 * (1 if case["bias"] == "sandwich" else Hq)
        factors = rows_k + rows_q
    return {"bytes": 2 * H * keys * held + B * Hq * T * (4 * d + 4) + tables + factors,
            "flops": pairs * (4 * d + 2 * R)}


def exact(case, seed):
    s = prepare(case, seed)
    f64, B, d = torch.float64, case["batch"], case["dim"]
    if case["op"] in ("rope", "rope_grad"):
        rot, out = case["rotary"], []
        half = rot // 2
        one, two = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, half), slice(half, rot))
        theta = torch.einsum("bn,k->bnk", s["positions"].to(f64), s["freq"])[:, None]
        if case["op"] == "rope_grad":
            theta = -theta
        z = torch.polar(torch.full_like(theta, s["factor"]), theta)
        for x in (s["q"], s["k"]):
            y = x.to(f64).clone()
            w = torch.complex(y[..., one], y[..., two]) * z
            y[..., one], y[..., two] = w.real, w.imag
            out.append(y)
        return out

    H, page = case["kv_heads"], case["page"]
    table = s["table"].tolist()

    def power(e):  # 2^e, from its bits
        return ((e.long() + 1023) << 52).view(f64)

    def held(name):  # the cache's values
        if case["cache"] != "e4m3":
            return s[name].to(f64)
        c = s[name].view(torch.uint8).long()
        e, m = (c >> 3) & 15, (c & 7).to(f64)
        x = torch.where(e > 0, (8 + m) * power(e - 10), m * 2.0 ** -9)
        x = torch.where(c > 127, -x, x)
        return x * power(s[name + "_scale"].view(torch.uint8).long() - 127)[..., None]

    if case["op"] == "write":
        out = []
        for name in ("k", "v"):
            pool, new = s[name].to(f64).clone(), s["new_" + name].to(f64)
            scales = None
            if case["cache"] == "e4m3":
                scales = s[name + "_scale"].to(torch.float32).to(f64).clone()
                top = new.abs().amax(-1)
                e = torch.ceil(torch.log2(top.clamp(min=1e-300) / E4M3_MAX)).clamp(min=-126)
                e = torch.where(top * power(-e) > E4M3_MAX, e + 1, e)
                e = torch.where((top * power(1 - e) <= E4M3_MAX) & (e > -126), e - 1, e)
                x = new * power(-e)[..., None]
                step = power(torch.frexp(x.abs().clamp(min=2.0 ** -6))[1] - 4)
                new = torch.round(x / step) * step
            elif case["type"] == "f32":
                new = s["new_" + name].to(torch.bfloat16).to(f64)
            for b, (first, n) in enumerate(zip(s["starts"].tolist(), s["counts"].tolist())):
                i = torch.arange(first, first + n)
                at = torch.tensor(table[b])[i // page].cuda()
                pool[at, :, (i % page).cuda()] = new[b, :, :n].transpose(0, 1)
                if scales is not None:
                    scales[at, :, (i % page).cuda()] = power(e)[b, :, :n].transpose(0, 1)
            out.append((pool, scales))
        return [x for x in (out[0][0], out[1][0], out[0][1], out[1][1]) if x is not None]

    def rows(x, b, n, first=0):  # [H, n, d] of sequence b
        i = torch.arange(first, first + n)
        return x[torch.tensor(table[b])[i // page].cuda(), :, (i % page).cuda()].transpose(0, 1)

    if case["op"] == "read":
        out = []
        for name in ("k", "v"):
            x, y = held(name), torch.zeros((B, H, case["tokens"], d), dtype=f64, device="cuda")
            for b, (first, n) in enumerate(zip(s["starts"].tolist(), s["counts"].tolist())):
                y[b, :, :n] = rows(x, b, n, first)
            out.append(y)
        return out

    k, v = held("k"), held("v")
    Hq, T, R = case["q_heads"], case["tokens"], case["rank"]
    o = torch.zeros((B, Hq, T, d), dtype=f64, device="cuda")
    lse = torch.full((B, Hq, T), -math.inf, dtype=f64, device="cuda")
    for b, (a, n) in enumerate(zip(s["prefix"].tolist(), s["counts"].tolist())):
        if n == 0:
            continue
        kb, vb = rows(k, b, a + n), rows(v, b, a + n)
        if case["tree"]:
            w = s["mask"][b, :n].cpu().numpy().view("uint32").tolist()
            see = torch.tensor([[bool(w[t][u // 32] >> (u % 32) & 1) for u in range(n)] for t in range(n)]).cuda()
            depth = s["depth"][b, :n].long()
        else:
            see, depth = torch.ones((n, n), dtype=torch.bool, device="cuda").tril(), torch.arange(n, device="cuda")
        see = torch.cat([torch.ones((n, a), dtype=torch.bool, device="cuda"), see], 1)
        kpos = torch.cat([torch.arange(a, device="cuda"), a + depth])
        for h in range(Hq):
            g = h // (Hq // H)
            x = s["q"][b, h, :n].to(f64) @ kb[g].T / math.sqrt(d)
            if R:
                fq, fk = s["phi_q"][min(h, len(s["phi_q"]) - 1)], s["phi_k"][min(g, len(s["phi_k"]) - 1)]
                x = x + fq[a + depth].to(f64) @ fk[kpos].to(f64).T
            x = x.masked_fill(~see, -math.inf)
            lse[b, h, :n] = torch.logsumexp(x, -1)
            o[b, h, :n] = torch.softmax(x, -1) @ vb[g]
    return [o, lse]
