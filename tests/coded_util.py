"""Plain float64 forms of the 8-bit cache, of norms with rotation, and of attention over codes, for their tests."""
import numpy as np
import torch

E4M3 = "e4m3"
INT8 = "int8"


def e4m3_values():
    """What the 256 codes of the 8-bit floating type stand for: 1 sign, 4 exponent (bias 7) and 3 mantissa bits."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = np.ldexp(1 + m / 8, e - 7) if e else np.ldexp(m / 8, -6)
        out[c] = np.nan if (c & 127) == 127 else (-v if c & 128 else v)
    return out


def quantise_ref(x, quant):
    """Vectors along the last axis (a CPU tensor of a 16-bit type): codes as
    uint8, scales as float32, and the values they stand for in float64.  A
    float32 product or quotient is formed in float64 and rounded, which is the
    same number (53 bits hold more than twice 24)."""
    x = x.double().numpy()
    top = np.abs(x).max(-1)
    finite = np.isfinite(x).all(-1)
    small = top < 2.0 ** -100
    ok = finite & ~small
    t = np.where(ok, top, 1.0)
    if quant == E4M3:
        n = np.ceil(np.log2(t / 448.0))
        n = np.where(448.0 * np.exp2(n - 1) >= t, n - 1, n)
        n = np.where(448.0 * np.exp2(n) < t, n + 1, n)
        scale = np.exp2(n)
        y = np.where(ok[..., None], x, 0) / scale[..., None]
        a = np.abs(y)
        step = np.exp2(np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
        q = np.rint(a / step) * step                                       # to even: multiples of the step
        mag = e4m3_values()[:127]
        codes = np.searchsorted(mag, q)
        assert (mag[codes] == q).all()
        codes = codes | (np.signbit(y) << 7)
        values = np.copysign(q, y)
    else:
        t32 = t.astype(np.float32)
        scale = (t32 / np.float32(127)).astype(np.float64)
        inv = np.float32(127) / t32
        y = (np.where(ok[..., None], x, 0).astype(np.float32) * inv[..., None])
        values = np.rint(y).astype(np.float64)
        codes = values.astype(np.int8).view(np.uint8).astype(np.int64)
    codes = np.where(ok[..., None], codes, 0)
    scale = np.where(finite, np.where(small, 0.0, scale), np.nan).astype(np.float32)
    values = np.where(ok[..., None], values, 0.0) * scale.astype(np.float64)[..., None]
    return torch.from_numpy(codes.astype(np.uint8)), torch.from_numpy(scale), torch.from_numpy(values)


def rope_ref(x, positions, inv_freq, weight=None, eps=1e-6, interleaved=False):
    """[rows, heads, D] in float64, and next to each number the size of the pair it came from."""
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps) * weight.double()
    R = 2 * inv_freq.numel()
    i = torch.arange(R // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    t = positions.double()[:, None, None] * inv_freq
    out, size = y.clone(), y.abs()
    out[..., a] = y[..., a] * t.cos() - y[..., b] * t.sin()
    out[..., b] = y[..., b] * t.cos() + y[..., a] * t.sin()
    size[..., a] = size[..., b] = y[..., a].abs() + y[..., b].abs()
    return out, size


def make_coded_pages(L, P, KV, D, dtype, quant, seed, extra=3):
    """serving_util.make_pages as codes: the pools on the GPU, and what they
    stand for as float64 pools for serving_util.attention_ref.  What no token
    fills holds codes that are no numbers and scales that are not finite."""
    from . import serving_util as su
    k, v, table, seq_len = su.make_pages(L, P, KV, D, dtype, seed, extra=extra)
    out, ref = [], []
    for t in (k, v):
        codes, scale, values = quantise_ref(t.cpu(), quant)
        empty = scale.isnan()
        codes[empty] = 0x7F
        scale[empty] = torch.tensor([torch.nan, torch.inf, -torch.inf, 0.0]).repeat(int(empty.sum()) // 4 + 1)[:int(empty.sum())]
        out += [codes.cuda().view(torch.float8_e4m3fn if quant == E4M3 else torch.int8), scale.cuda()]
        ref.append(values)
    return out, ref, table, seq_len


def make_shared(groups, P, KV, D, dtype, quant, seed, extra=3):
    """Sequences that were forked off their group's prefix: groups is a list of
    (prefix length, [own tokens of each member]).  Whole pages of a prefix are
    shared, a partly filled last one is copied for every member but the first.
    Returns pools (k, k_scale, v, v_scale; scales None without quant), float64
    pools, page_table, seq_len, groups and prefix_len."""
    g = torch.Generator().manual_seed(seed)
    tables, copies, fill, n = [], [], [], 0
    for prefix, own in groups:
        whole = list(range(n, n + prefix // P))
        n += len(whole)
        for m, o in enumerate(own):
            L = prefix + o
            mine = list(range(n, n + -(-L // P) - len(whole)))
            n += len(mine)
            if prefix % P and m:
                copies.append((lead, mine[0], prefix % P))
            elif prefix % P:
                lead = mine[0]
            tables.append(whole + mine)
            fill.append((tables[-1][-1] if L % P else None, L % P))
    total = n + extra
    ids = torch.randperm(total, generator=g)
    pools = []
    for _ in range(2):
        x = torch.randn(total, KV, P, D, generator=g).to(dtype)
        for src, dst, c in copies:
            x[dst, :, :c] = x[src, :, :c]
        for page, c in fill:
            if page is not None:
                x[page, :, c:] = torch.nan
        x[n:] = torch.nan
        out = torch.empty_like(x)
        out[ids] = x
        pools.append(out)
    width = max(len(t) for t in tables)
    table = torch.full((len(tables), max(width, 1)), -1, dtype=torch.int32)
    for b, t in enumerate(tables):
        table[b, :len(t)] = ids[torch.tensor(t, dtype=torch.int64)].to(torch.int32)
    dev, ref = [], []
    for x in pools:
        if quant is None:
            dev += [x.cuda(), None]
            ref.append(x.double())
        else:
            codes, scale, values = quantise_ref(x, quant)
            codes[scale.isnan()] = 0x7F
            dev += [codes.cuda().view(torch.float8_e4m3fn if quant == E4M3 else torch.int8), scale.cuda()]
            ref.append(values)
    first = np.cumsum([0] + [len(own) for _, own in groups])
    L = [p + o for p, own in groups for o in own]

    def i32(x):
        return torch.tensor(x, dtype=torch.int32).cuda()
    return dev, ref, table.cuda(), i32(L), i32(first.tolist()), i32([p for p, _ in groups])


def ramp_keys(pools, ref, table, seq_len, P, quant, falling=False, top=3.0):
    """The first number of every key becomes 0 .. top by its position (or top ..
    0), in the pools and in what they stand for: scores that grow or fall."""
    L = int(seq_len.max())
    table, k = table.cpu().long(), pools[0].cpu()
    for b, n in enumerate(seq_len.tolist()):
        pos = torch.arange(n)
        page, off = table[b, pos // P], pos % P
        r = ((L - 1 - pos if falling else pos).double() * (top / L))[:, None]
        if quant is None:
            v = r.to(k.dtype).expand(n, k.shape[1])
            k[page, :, off, 0] = v
            ref[0][page, :, off, 0] = v.double()
        else:
            s = pools[1].cpu()[page, :, off].double()
            if quant == E4M3:
                c = (r / s).clamp(max=448.0).to(torch.float8_e4m3fn)
                k.view(torch.uint8)[page, :, off, 0] = c.view(torch.uint8)
            else:
                c = (r / s).clamp(max=127.0).round().to(torch.int8)
                k[page, :, off, 0] = c
            ref[0][page, :, off, 0] = c.double() * s
    pools[0].copy_(k)
