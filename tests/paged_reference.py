"""Plain 64-bit implementations of the serving operators, for the tests, on the CPU.

They share nothing with the kernels.  The attention reference also returns what its
tolerance needs: the weighted mean of |v| and a bound on the fp32 error of a row's scores.
"""
import math

import torch

BF16_HALF_STEP = 2.0 ** -8     # rounding to bf16, relative to the value


def rope(x, weight, positions, inv_freq, eps, interleaved, factor):
    """x [..., T, D] with positions [..., T] broadcast against it: (result, magnitude of each element's pair)."""
    y = x.double()
    D = y.shape[-1]
    if weight is not None:
        y = y / (y.pow(2).mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    mag = y.abs()
    if inv_freq is None:
        return y, mag
    n = inv_freq.numel()
    i = torch.arange(n)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    t = positions.double()[..., None] * inv_freq
    c, s = t.cos() * factor, t.sin() * factor
    out = y.clone()
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., b] * c + y[..., a] * s
    mag = mag.clone()
    mag[..., a] = mag[..., b] = torch.hypot(y[..., a], y[..., b]) * abs(factor)
    return out, mag


def e4m3_table():
    """The value of each of the 256 codes."""
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.nan if (e, m) == (15, 7) else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v.append(-x if c & 128 else x)
    return torch.tensor(v, dtype=torch.float64)


def quantise(rows):
    """rows [..., D] bf16 -> (codes uint8 [..., D], scale codes uint8 [...]) by searching the e4m3 table."""
    x = rows.double()
    flat = x.reshape(-1, x.shape[-1])
    codes = torch.empty(flat.shape, dtype=torch.uint8)
    scales = torch.empty(flat.shape[0], dtype=torch.uint8)
    pos = e4m3_table()[:127]                       # 0 .. 448, ascending
    for r in range(flat.shape[0]):
        row = flat[r]
        if not torch.isfinite(row).all():
            codes[r], scales[r] = 0x7F, 255
            continue
        amax = row.abs().max().item()
        e = 0
        if amax > 0:
            e = -117
            while amax / 2.0 ** e > 448.0 and e < 120:
                e += 1
        z = row / 2.0 ** e
        a = z.abs().clamp(max=240.0 if e == 120 else 448.0)      # 256 * 2^120 would be infinite in bf16
        hi = torch.searchsorted(pos, a).clamp(1, 126)
        lo = hi - 1
        d_lo, d_hi = a - pos[lo], pos[hi] - a
        near = torch.where((d_hi < d_lo) | ((d_hi == d_lo) & (hi % 2 == 0)), hi, lo)   # ties to the even code
        codes[r] = (near + torch.where(torch.signbit(z), 128, 0)).to(torch.uint8)
        scales[r] = e + 127
    return codes.reshape(x.shape), scales.reshape(x.shape[:-1])


def dequantise(codes, scales):
    s = torch.where(scales == 255, math.nan, 2.0 ** (scales.double() - 127))
    return e4m3_table()[codes.long()] * s[..., None]


def gather(pages, table_row, n):
    """[Hkv, n, D]: the first n rows of one sequence; a page outside the pool reads as zeros."""
    P, H, page, D = pages.shape
    out = torch.zeros(H, n, D, dtype=torch.float64)
    for j in range(0, n, page):
        pg = int(table_row[j // page])
        m = min(page, n - j)
        if 0 <= pg < P:
            out[:, j:j + m] = pages[pg, :, :m].double()
    return out


def paged(q, k_pages, v_pages, table, kv_len, q_start, causal, scale):
    """Everything on the CPU; pages as values.  Returns (out, lse, mean |v|, score error bound), rows
    outside every sequence NaN."""
    T, Hq, D = q.shape
    G = Hq // k_pages.shape[1]
    out = torch.full((T, Hq, D), math.nan, dtype=torch.float64)
    mean = out.clone()
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64)
    err = torch.zeros((T, Hq), dtype=torch.float64)
    for b, n in enumerate(kv_len):
        t0, t1 = q_start[b], q_start[b + 1]
        k = gather(k_pages, table[b], n).repeat_interleave(G, 0)
        v = gather(v_pages, table[b], n).repeat_interleave(G, 0)
        qb = q[t0:t1].double().transpose(0, 1)                       # [Hq, n_q, D]
        s = qb @ k.transpose(1, 2) * scale
        if causal:
            last = torch.arange(t1 - t0)[:, None] + n - (t1 - t0)
            s = s.masked_fill(torch.arange(n) > last, -math.inf)
        if n:
            m = s.amax(-1, keepdim=True)
            dead = m == -math.inf
            p = torch.where(dead, 0.0, (s - torch.where(dead, 0.0, m)).exp())
            l = p.sum(-1, keepdim=True)
            p = p / torch.where(l == 0, 1.0, l)
            out[t0:t1] = (p @ v).transpose(0, 1)
            mean[t0:t1] = (p @ v.abs()).transpose(0, 1)
            lse[t0:t1] = torch.where(dead, -math.inf, m + l.log())[..., 0].T
            worst = (qb.abs() @ k.abs().transpose(1, 2)).amax(-1) * abs(scale)
            err[t0:t1] = ((D + 4) * 2.0 ** -24 * worst).T
        else:
            out[t0:t1], mean[t0:t1], lse[t0:t1] = 0.0, 0.0, -math.inf
    return out, lse, mean, err


def assert_paged_close(out, lse, ref):
    """Tolerances: an fp32 score is off by at most `err` (D + 4 roundings of 2^-24 on the sum of
    |q||k|), and ex2 by 2^-21, so each weight by err' = 2 err + 2^-20 relative to the weight sum (numerator
    and denominator); a weight is rounded to bf16 (half a step) and so is the result; the row sum of n
    fp32 terms adds at most n 2^-24, taken as 2^-9 for the sizes tested (n <= 32768)."""
    r_out, r_lse, mean, err = ref
    out, lse = out.detach().cpu().double(), lse.detach().cpu().double()
    live = ~torch.isnan(r_lse)
    e = 2 * err + 2.0 ** -20
    tol = mean * (BF16_HALF_STEP * 1.01 + e[..., None] + 2.0 ** -9) + BF16_HALF_STEP * r_out.abs() + 1e-30
    bad = (~((out - r_out).abs() <= tol))[live]
    assert not bad.any(), f"out: {int(bad.sum())} of {bad.numel()} off, worst {((out - r_out).abs() / tol)[live].max():.3g} of the tolerance"
    dead = live & (r_lse == -math.inf)
    assert (lse[dead] == -math.inf).all() and (out[dead] == 0).all(), "empty rows"
    some = live & ~dead
    d = (lse - r_lse).abs()[some]
    tol = (err + 2.0 ** -20 * (1 + r_lse.abs()) + 2.0 ** -9)[some]
    assert (d <= tol).all(), f"lse: worst {(d / tol).max():.3g} of the tolerance"
