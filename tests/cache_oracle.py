"""FP64 oracle of the paged cache (plain loops over sequences, heads and pages)
and the bounds that the kernels' results are held to."""
from __future__ import annotations

import torch

E4M3_MAX = 448.0


def page_rows(pages, scale, table_row, head, n):
    """The first n tokens of one head of a sequence, FP64, from pages
    [num_pages, page_size, heads, 128]; a page number outside the pool reads
    as zeros."""
    page_size = pages.shape[1]
    out = torch.zeros(n, pages.shape[3], dtype=torch.float64)
    for j0 in range(0, n, page_size):
        pid = int(table_row[j0 // page_size])
        m = min(page_size, n - j0)
        if 0 <= pid < pages.shape[0]:
            x = pages[pid, :m, head].double()
            out[j0:j0 + m] = x * (1.0 if scale is None else float(scale[pid, head]))
    return out


def attend(q, k_pages, v_pages, k_scale, v_scale, table, seqlens, news, causal, window, scale):
    """(O [rows, h_q, 128], LSE [h_q, rows], bound of |dO|, bound of |dLSE|).

    Bounds, by the roundings that the kernel makes (u = 2^-8, half a step of
    BF16):
      - O is rounded to BF16: u |O|;
      - a weight is rounded to BF16, or to FP16 and then to nine bits
        (2^-11 + 2^-9 < u), with a floor of 2^-27 of the row's unit, which is
        at most twice the largest weight: (u P + 2^-26 max P) |V|, summed;
      - a score is off by `ds`: FP32 sums of 128 products (2^-17 of the sum of
        |q k|), the part of Q below two E4M3 numbers (2^-17 of the row's
        largest |q| times the sum of |k|), and the rounding of the exponent
        (FP32 at up to 2^7 + |s|) and of ex2 (2^-22): each weight moves by a
        factor 1 + ds at most, and so does their sum.
    """
    rows, h_q = q.shape[0], q.shape[1]
    h_kv, cap = k_pages.shape[2], table.shape[1] * k_pages.shape[1]
    o = torch.zeros(rows, h_q, 128, dtype=torch.float64)
    lse = torch.full((h_q, rows), float("-inf"), dtype=torch.float64)
    do, dl = torch.zeros_like(o), torch.zeros_like(lse)
    u, row = 2.0 ** -8, 0
    for b, (length, n) in enumerate(zip(seqlens, news)):
        keys = max(0, min(length, cap))
        for h in range(h_kv if n else 0):
            k = page_rows(k_pages, k_scale, table[b], h, keys)
            v = page_rows(v_pages, v_scale, table[b], h, keys)
            j = torch.arange(keys)
            for e in range(h * (h_q // h_kv), (h + 1) * (h_q // h_kv)):
                x = q[row:row + n, e].double()
                s = x @ k.T * scale
                off = abs(scale) * (2.0 ** -17 * (x.abs() @ k.abs().T) + 2.0 ** -17 *
                                    x.abs().amax(-1, keepdim=True) * k.abs().sum(-1)[None])
                off = off + 2.0 ** -17 + 2.0 ** -23 * s.abs()
                for i in range(n):
                    last = length - n + i
                    seen = j <= last if causal else torch.ones(keys, dtype=torch.bool)
                    if window >= 0:
                        seen &= j >= last - window
                    if not seen.any():
                        continue
                    y, w = s[i, seen], v[seen]
                    p = torch.softmax(y, 0)
                    o[row + i, e] = p @ w
                    lse[e, row + i] = torch.logsumexp(y, 0)
                    ds = float(off[i, seen].max())
                    do[row + i, e] = (u * o[row + i, e].abs() + (u + 3 * ds) * (p @ w.abs()) +
                                      2.0 ** -26 * p.max() * w.abs().sum(0) + 1e-30)
                    dl[e, row + i] = 2 * ds + 2.0 ** -21 * (1 + abs(float(lse[e, row + i])))
        row += n
    return o, lse, do, dl


def assert_attend(o, lse, ref):
    ro, rl, do, dl = ref
    o, lse = o.cpu().double()[:ro.shape[0]], lse.cpu().double()[:, :rl.shape[1]]
    assert torch.equal(torch.isinf(lse), torch.isinf(rl))
    assert bool((lse[torch.isinf(rl)] < 0).all())
    bad = (o - ro).abs() - do
    assert float(bad.max()) <= 0, f"O off by {float((o - ro).abs().max()):.3e}, {int((bad > 0).sum())} values"
    fin = torch.isfinite(rl)
    if fin.any():
        off = (lse - rl)[fin].abs() - dl[fin]
        assert float(off.max()) <= 0, f"LSE off by {float((lse - rl)[fin].abs().max()):.3e}"


def rotate(x, first, inv_freq, interleaved):
    """x [rows, heads, 128] FP64, row i at position first + i."""
    if inv_freq is None:
        return x.clone()
    half = inv_freq.numel()
    angle = (first + torch.arange(x.shape[0], dtype=torch.float64))[:, None] * inv_freq.double()
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    y = x.clone()
    i0 = torch.arange(half) * 2 if interleaved else torch.arange(half)
    i1 = i0 + (1 if interleaved else half)
    y[..., i0] = x[..., i0] * c - x[..., i1] * s
    y[..., i1] = x[..., i1] * c + x[..., i0] * s
    return y


def pow2_scale(bound):
    """The smallest power of two s with bound <= 448 s, 0 for 0."""
    if bound == 0:
        return 0.0
    s = 2.0 ** -140
    while bound > E4M3_MAX * s:
        s *= 2
    return max(s, 2.0 ** -126)


def append(k, v, k_pages, v_pages, k_scale, v_scale, table, seqlens, news, inv_freq, interleaved):
    """What the pool holds after the call: (values of k, values of v, k_scale,
    v_scale, written).  Values are FP64 and unrounded for the new rows; older
    rows are the pool's codes times their factor; `written` [num_pages,
    page_size] is 2 for new rows, 1 for rows of a page and head that was coded
    again, 0 elsewhere."""
    page_size, h_kv = k_pages.shape[1], k_pages.shape[2]
    cap = table.shape[1] * page_size
    vals = [k_pages.double().clone(), v_pages.double().clone()]
    e4m3 = k_scale is not None
    scales = [k_scale.double().clone(), v_scale.double().clone()] if e4m3 else [None, None]
    written = torch.zeros(k_pages.shape[:2], dtype=torch.int64)
    row = 0
    half = 0 if inv_freq is None else inv_freq.numel()
    for b, (length, n) in enumerate(zip(seqlens, news)):
        first = length - n
        turned = (rotate(k[row:row + n].double(), first, inv_freq, interleaved),
                  v[row:row + n].double())
        plain = (k[row:row + n].double(), v[row:row + n].double())
        row += n
        lo, hi = max(first, 0), min(length, cap)
        for page in range(lo // page_size, (hi - 1) // page_size + 1 if hi > lo else 0):
            pid = int(table[b, page])
            if not 0 <= pid < k_pages.shape[0]:
                continue
            a, z = max(lo, page * page_size), min(hi, (page + 1) * page_size)
            s0, rows = a - page * page_size, slice(a - first, z - first)
            for t in range(2):
                if e4m3:
                    top = plain[t][rows].abs()
                    if t == 0 and half:
                        i0 = torch.arange(half) * 2 if interleaved else torch.arange(half)
                        i1 = i0 + (1 if interleaved else half)
                        # FP32, as a BF16 sum that needs more bits is rounded
                        pair = (top[..., i0].float() + top[..., i1].float()).double()
                        top = torch.cat((pair, top[..., 2 * half:]), -1)
                    for h in range(h_kv):
                        old = float(scales[t][pid, h]) if s0 > 0 else 0.0
                        new = max(old, pow2_scale(float(top[:, h].max())))
                        if s0 > 0 and new > old > 0:
                            vals[t][pid, :s0, h] *= old / new
                        scales[t][pid, h] = new
                        vals[t][pid, s0:s0 + z - a, h] = turned[t][rows, h] / (new or 1.0)
                else:
                    vals[t][pid, s0:s0 + z - a] = turned[t][rows]
            written[pid, s0:s0 + z - a] = 2
            if e4m3 and s0 > 0:
                written[pid, :s0] = torch.maximum(written[pid, :s0],
                                                  torch.ones(s0, dtype=torch.int64))
    return vals[0], vals[1], scales[0], scales[1], written


def assert_pages(got, want, e4m3, written, before):
    """Pages against the oracle's values: a new value is rounded once (half a
    step of E4M3: 2^-4 of it, 2^-10 where subnormal; of BF16 2^-8) after an FP32
    rotation (2^-21 of the pair, whose length is at most 448 of the scale, or
    sqrt 2 times the largest value); an older one coded again likewise; rows
    that the call does not write keep their bits."""
    got, want = got.cpu(), want
    same = written == 0
    bits = torch.uint8 if e4m3 else torch.int16
    assert torch.equal(got[same].contiguous().view(bits), before[same].contiguous().view(bits))
    g, w = got[~same].double(), want[~same]
    if not g.numel():
        return
    if e4m3:
        bound = 2.0 ** -4 * w.abs() + 2.0 ** -10 + 2.0 ** -21 * 448
    else:
        bound = 2.0 ** -8 * w.abs() + 2.0 ** -20 * w.abs().max()
    bad = (g - w).abs() - bound
    assert float(bad.max()) <= 0, f"off by {float((g - w).abs().max()):.3e}"
