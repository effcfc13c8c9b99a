"""Plain 64-bit implementations of the serving operators (rotary positions, the
paged cache, attention over it), and error bounds for the kernels, shared by
their tests. Everything here is elementary torch on the CPU."""
import math

import torch

F64 = torch.float64


def rope(x, freq, positions, rot, interleaved, factor=1.0, sign=1.0):
    """x [B, H, N, d]; positions [B, N]."""
    y = x.to(F64).clone()
    ang = sign * positions.to(F64)[:, None, :, None] * torch.tensor(freq, dtype=F64)
    c, s = factor * ang.cos(), factor * ang.sin()
    ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    a, b = x.to(F64)[..., ia], x.to(F64)[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    return y


def e4m3_values(codes):
    """Values of e4m3 codes (uint8), NaN for 0x7f and 0xff."""
    c = codes.to(torch.int64)
    e, m = (c >> 3) & 15, (c & 7).to(F64)
    x = torch.where(e > 0, (8 + m) * 2.0 ** (e.to(F64) - 10), m * 2.0 ** -9)
    x = torch.where((c & 127) == 127, torch.full_like(x, math.nan), x)
    return torch.where(c > 127, -x, x)


def quantise(x):
    """(codes uint8, scale bytes uint8) of the rows of x: the least power of two from 2^-126 that brings the largest
    finite value to 448 or less, then the nearest e4m3 value (ties to the even code), searched among all of them."""
    x = x.to(F64)
    top = torch.where(x.isfinite(), x.abs(), torch.zeros_like(x)).amax(-1)
    e = torch.full(top.shape, -126, dtype=torch.int64)
    while True:
        up = top > 448.0 * 2.0 ** e.to(F64)
        if not up.any():
            break
        e = e + up.long()
    y = x * 2.0 ** -e.to(F64)[..., None]
    table = e4m3_values(torch.arange(127, dtype=torch.uint8))  # ascending, code = index
    mag = y.abs().nan_to_num(0.0, posinf=448.0).clamp(max=448.0)
    hi = torch.searchsorted(table, mag.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = mag - table[lo], table[hi] - mag
    pick = torch.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    pick = torch.where(y.isnan(), torch.full_like(pick, 127), pick)
    codes = (pick + 128 * torch.signbit(y).long()).to(torch.uint8)
    return codes, (e + 127).to(torch.uint8)


def pool_values(pool, scale=None):
    """[pages, H, page, d] in 64 bits."""
    if scale is None:
        return pool.to(F64)
    return e4m3_values(pool.view(torch.uint8)) * 2.0 ** (scale.view(torch.uint8).to(F64) - 127)[..., None]


def rows(values, table, first, count):
    """Tokens first .. first + count - 1 of one sequence: [H, count, d]."""
    page = values.shape[2]
    i = torch.arange(first, first + count)
    return values[table[i // page].long(), :, i % page].transpose(0, 1)


def visible(mask, T, n, b):
    """[n, n] truth values: new token t sees new token u."""
    if mask is None:
        return torch.ones(n, n, dtype=torch.bool).tril()
    w = mask[b].to(torch.int64) & 0xFFFFFFFF
    u = torch.arange(n)
    return ((w[:n][:, u // 32] >> (u % 32)) & 1).bool()


def attend(q, kv, vv, table, prefix, counts, mask=None, depths=None, phi_q=None, phi_k=None, scale=None, part_bits=8):
    """O, LSE and bounds on their errors, [B, Hq, T, d] and [B, Hq, T].

    kv, vv: the pools' values in 64 bits. part_bits: a probability is off by at
    most 2^-part_bits of itself for the product with V (bf16 8, fp16 11).

    The bounds: scores are sums in fp32 of d exact products (each addition
    rounds to 2^-24 of the running magnitude, which tensor cores may truncate:
    2^-23), then one scaling and one addition of the bias. A bias of rank R up
    to 4 is R fp32 multiply-adds. A larger one is 3 R products of 22-bit parts:
    a part pair is off by 2^-22 of the value, or by 2^-25 of its column's balanced
    size, the dropped low product by 2^-22, the sum by 3 R 2^-23. exp2 is good to
    2^-22 and its argument rounds to 2^-24 of |x - max| log2 e, at most 150."""
    B, Hq, T, d = q.shape
    H = kv.shape[1]
    scale = d ** -0.5 if scale is None else scale
    o, lse = torch.zeros(B, Hq, T, d, dtype=F64), torch.full((B, Hq, T), -math.inf, dtype=F64)
    o_tol, lse_tol = torch.zeros_like(o), torch.zeros(B, Hq, T, dtype=F64)
    for b in range(B):
        a, n = int(prefix[b]), int(counts[b])
        if n == 0:
            continue
        k, v = rows(kv, table[b], 0, a + n), rows(vv, table[b], 0, a + n)
        see = torch.cat([torch.ones(n, a, dtype=torch.bool), visible(mask, T, n, b)], 1)
        depth = torch.arange(n) if depths is None else depths[b, :n].long()
        kpos = torch.cat([torch.arange(a), a + depth])
        for h in range(Hq):
            g = h // (Hq // H)
            qh = q[b, h, :n].to(F64)
            x = scale * qh @ k[g].T
            dx = ((d + 4) * 2.0 ** -23) * scale * (qh.abs() @ k[g].abs().T)
            if phi_q is not None:
                fq, fk = phi_q[min(h, phi_q.shape[0] - 1)], phi_k[min(g, phi_k.shape[0] - 1)]
                R = fq.shape[-1]
                fq, fk = fq[a + depth].to(F64), fk[kpos].to(F64)
                x = x + fq @ fk.T
                size = fq.abs() @ fk.abs().T
                if R <= 4:
                    dx = dx + 2.0 ** -21 * size
                else:
                    col = phi_q.abs().amax((0, 1)).to(F64) * phi_k.abs().amax((0, 1)).to(F64)
                    dx = dx + (3 * 2.0 ** -22 + 3 * R * 2.0 ** -23) * size + 2 * 2.0 ** -24 * col.sqrt().sum() * max(
                        1.0, float(col.max()) ** 0.5)
            dx = (dx + 2.0 ** -23 * x.abs()).masked_fill(~see, 0.0)
            x = x.masked_fill(~see, -math.inf)
            lse[b, h, :n] = torch.logsumexp(x, -1)
            p = torch.softmax(x, -1).nan_to_num(0.0)
            vg = torch.where(see[..., None], v[g][None], torch.zeros(1, dtype=F64)) if not v[g].isfinite().all() else None
            if vg is None:
                o[b, h, :n] = p @ v[g]
                weight = p @ v[g].abs()
            else:
                o[b, h, :n] = torch.einsum("tj,tjd->td", p, vg)
                weight = torch.einsum("tj,tjd->td", p, vg.abs())
            step = dx.amax(-1) + 2.0 ** -16  # 150 * 2^-24 * ln 2 and exp2, rounded up
            lse_tol[b, h, :n] = step + 2.0 ** -22 * lse[b, h, :n].abs().nan_to_num(0.0, posinf=0.0)
            o_tol[b, h, :n] = 2.0 ** -8 * o[b, h, :n].abs() + (2.0 ** -part_bits + 2 * step[:, None]) * weight
    return o, lse, o_tol, lse_tol
