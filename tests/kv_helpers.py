"""Plain CPU forms of the rotary append, of the attention over the paged E4M3
cache and of the bf16-activation linear, in 64 bits (and, for the append, also
step by step in binary32, which the kernel has to match bit for bit), and the
batches that the tests run them on."""
import math

import torch

E_MIN, E_MAX = -96, 119


def e4m3(v):
    """RNE onto E4M3, saturating (torch's cast alone turns overflow into NaN)."""
    return v.clamp(-448.0, 448.0).float().to(torch.float8_e4m3fn)


def exponent(amax):
    """Least e with amax <= 448 * 2^e, in [E_MIN, E_MAX]; a Python float's."""
    if not amax > 0:
        return E_MIN
    m, x = math.frexp(amax)
    return min(E_MAX, max(E_MIN, x - 9 if m <= 0.875 else x - 8))


def rope(positions, rot_dim, theta=1e4):
    f = theta ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def rotate(x, cs, rot_dim, interleaved):
    """x [heads, D] at one position, cs its table row; every step one operation of x's type."""
    out = x.clone()
    h = rot_dim // 2
    c, s = cs[:h].to(x.dtype), cs[h:rot_dim].to(x.dtype)
    ia = torch.arange(h) * 2 if interleaved else torch.arange(h)
    ib = ia + (1 if interleaved else h)
    a, b = x[:, ia], x[:, ib]
    out[:, ia] = a * c - b * s
    out[:, ib] = b * c + a * s
    return out


class Batch:
    """Sequences (new tokens, length with them) on a pool of pages in random order, with the tables as the calls
    take them; codes and scales of every page are filled with junk, 0x7F codes (NaN) among it."""

    def __init__(self, seqs, page, kv_heads, head_dim, seed=0, extra_rows=0, extra_pages=2):
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.page, self.H, self.D, self.g = seqs, page, kv_heads, head_dim, g
        used = [max(0, -(-length // page)) for _, length in seqs]
        self.pages = sum(used) + extra_pages
        order = torch.randperm(self.pages, generator=g).to(torch.int32)
        self.table = torch.full((len(seqs), max(1, max(used))), -7, dtype=torch.int32)
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = order[at:at + u]
            at += u
        self.cu = torch.tensor([0] + [n for n, _ in seqs], dtype=torch.int32).cumsum(0).to(torch.int32)
        self.lens = torch.tensor([length for _, length in seqs], dtype=torch.int32)
        self.T = int(self.cu[-1]) + extra_rows
        shape = (self.pages, kv_heads, page, head_dim)
        self.k = torch.randint(0, 256, shape, generator=g, dtype=torch.uint8)
        self.v = torch.randint(0, 256, shape, generator=g, dtype=torch.uint8)
        self.k[:, :, :, 0] = 0x7F
        self.v[:, :, :, -1] = 0x7F
        self.ks = torch.full((self.pages, kv_heads), 3.0e38)
        self.vs = torch.full((self.pages, kv_heads), 3.0e38)
        self.max_q = max(1, max(n for n, _ in seqs))
        self.max_len = max(0, max(length for _, length in seqs))

    def fill(self, k_size=1.0, v_size=1.0, spread=0):
        """Values for every token already cached or to be attended to: random, quantized page by page;
        `spread`: pages differ by up to 2^spread in size."""
        for b, (n, length) in enumerate(self.seqs):
            for i in range(max(0, -(-length // self.page))):
                p, m = int(self.table[b, i]), min(self.page, length - i * self.page)
                for codes, scales, size in ((self.k, self.ks, k_size), (self.v, self.vs, v_size)):
                    x = torch.randn(self.H, m, self.D, generator=self.g) * size
                    x *= 2.0 ** int(torch.randint(-spread, spread + 1, (1,), generator=self.g)) if codes is self.v else 1.0
                    for h in range(self.H):
                        s = 2.0 ** exponent(float(x[h].abs().max()))
                        scales[p, h] = s
                        codes[p, h, :m] = e4m3(x[h] / s).view(torch.uint8)
        return self

    def to(self, dev):
        f8 = torch.float8_e4m3fn
        return dict(cu_rows=self.cu.to(dev), lens=self.lens.to(dev), page_table=self.table.to(dev),
                    k_codes=self.k.to(dev).view(f8), v_codes=self.v.to(dev).view(f8), k_scales=self.ks.to(dev),
                    v_scales=self.vs.to(dev))

    def values(self, b, h):
        """k, v [length, D] of a sequence's kv head in 64 bits."""
        length = self.seqs[b][1]
        pg = self.table[b, :-(-length // self.page)].long()
        out = []
        for codes, scales in ((self.k, self.ks), (self.v, self.vs)):
            x = codes[pg, h].view(torch.float8_e4m3fn).double() * scales[pg, h].double()[:, None, None]
            out.append(x.reshape(-1, self.D)[:length])
        return out


def append_plain(bt, qkv, table, q_heads, rot_dim, interleaved, dtype):
    """The append on the batch's own tensors (in place); returns q [T, q_heads, D] in `dtype` (not rounded),
    NaN where a row is nobody's."""
    H, D, P = bt.H, bt.D, bt.page
    x = qkv.to(dtype).view(bt.T, q_heads + 2 * H, D)
    q = torch.full((bt.T, q_heads, D), math.nan, dtype=dtype)
    for b, (n, length) in enumerate(bt.seqs):
        r0 = int(bt.cu[b])
        rows = [(r0 + i, length - n + i) for i in range(n) if length - n + i >= 0]
        for r, pos in rows:
            cs = table[pos] if rot_dim else None
            q[r] = rotate(x[r, :q_heads], cs, rot_dim, interleaved) if rot_dim else x[r, :q_heads]
        by_page = {}
        for r, pos in rows:
            by_page.setdefault(pos // P, []).append((r, pos))
        for pi, members in by_page.items():
            p, first = int(bt.table[b, pi]), members[0][1] % P
            kk = torch.stack([rotate(x[r, q_heads:q_heads + H], table[pos], rot_dim, interleaved) if rot_dim
                              else x[r, q_heads:q_heads + H] for r, pos in members])      # [m, H, D]
            vv = torch.stack([x[r, q_heads + H:] for r, pos in members])
            for codes, scales, new in ((bt.k, bt.ks, kk), (bt.v, bt.vs, vv)):
                for h in range(H):
                    s = 2.0 ** exponent(float(new[:, h].abs().max()))
                    if first:
                        old = float(scales[p, h])
                        s = max(s, old)
                        if s > old:
                            c = codes[p, h, :first].view(torch.float8_e4m3fn).double() * (old / s)
                            codes[p, h, :first] = e4m3(c).view(torch.uint8)
                    scales[p, h] = s
                    codes[p, h, first:first + len(members)] = e4m3(new[:, h] / s).view(torch.uint8)
    return q


def attention_plain(bt, q, scale):
    """(out, bound) [T, q_heads, D] in 64 bits; rows that are nobody's are NaN.  `bound`: how far an output of the
    kernel may be from `out` before its own rounding to bf16.

    In units of 2^-24 = u (half a binary32 step, relative): a score s = scale sum q k is a binary32 sum of D exact
    products, in any order, truncated or rounded (2 u each): off by at most 2 (D + 4) u S, S = scale sum |q k|, the
    factors and the subtraction of the maximum included with |s| <= S; a weight's relative error is that, twice
    (its row's maximum), plus 2^-12 (its rounding to f16) and 2^-18 (the exponential: a polynomial
    within 2^-18.4, or ex2.approx within 2^-22; merges).  Sums over L keys
    add 2 L u.  A weight below f16's normal range is off by 2^-25 where the largest is at least 2^6, times a code
    of at most 448 under the largest scale.  q in f16 is exact above 2^-38 of its row's maximum, which the
    subnormal bound covers (D 2^-38 S)."""
    Hq, H, D = q.shape[1], bt.H, bt.D
    G = Hq // H
    u = 2.0 ** -24
    out = torch.full(q.shape, math.nan, dtype=torch.float64)
    bound = torch.zeros(q.shape, dtype=torch.float64)
    for b, (n, length) in enumerate(bt.seqs):
        r0 = int(bt.cu[b])
        if not n:
            continue
        if length <= 0:
            out[r0:r0 + n] = 0
            continue
        pos = torch.arange(length - n, length)
        hidden = torch.arange(length)[None, :] > pos[:, None]                       # [n, length]
        top_scale = float(bt.vs[bt.table[b, :-(-length // bt.page)].long()].max())
        for h in range(H):
            k, v = bt.values(b, h)
            for g in range(G):
                x = q[r0:r0 + n, h * G + g].double()
                s = (x @ k.T * scale).masked_fill(hidden, -math.inf)
                m = s.amax(1, keepdim=True).clamp(min=-1e300)
                w = (s - m).exp()
                w /= w.sum(1, keepdim=True).clamp(min=1e-300)
                S = (x.abs() @ k.abs().T * scale).masked_fill(hidden, 0).amax(1, keepdim=True)
                rel = 2 * (2 * (D + 4) * u + D * 2.0 ** -38) * S + 2.0 ** -12 + 2.0 ** -18 + 4 * length * u
                out[r0:r0 + n, h * G + g] = w @ v
                bound[r0:r0 + n, h * G + g] = 2 * rel * (w @ v.abs()) + length * 2.0 ** -31 * 448 * top_scale
    return out, bound


def close_to(got, want, bound, eps=2.0 ** -8):
    """Every |got - want| <= eps |want| + (1 + 2 eps) bound: bf16's rounding is off by half a step, 2^-8."""
    got, want = got.double(), want.double()
    err, most = (got - want).abs(), eps * want.abs() + (1 + 2 * eps) * bound + 1e-38
    worst = float((err / most).max())
    assert torch.isfinite(got).all() and worst <= 1.0, worst
    return worst


def nvfp4_values(codes, scales, alpha, N, K):
    """W [N, K] in 64 bits from the stored codes and MMA-ordered scales (uint8 tensors), alpha left out."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
    grid = torch.cat([grid, -grid])
    c = codes.view(N, K // 2)
    w = torch.stack([grid[(c & 15).long()], grid[(c >> 4).long()]], -1).view(N, K // 16, 16)
    r, kb = torch.arange(N)[:, None], torch.arange(K // 16)[None, :]
    at = (r // 128 * (K // 64) + kb // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + kb % 4
    return (w * scales.view(torch.float8_e4m3fn).double()[at][:, :, None]).view(N, K)
