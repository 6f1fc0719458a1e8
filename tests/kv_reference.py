"""Plain 64-bit statements of the K/V cache operators, for the tests: caches as torch tensors on any
device, one sequence at a time."""
from __future__ import annotations

import math

import torch

SIXTEEN = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # largest relative rounding error


def codes(packed: torch.Tensor) -> torch.Tensor:
    """Words [..., n] -> codes [..., 8 n] (little-endian nibbles)."""
    w = packed.long() & 0xFFFFFFFF
    return torch.stack([(w >> (4 * i)) & 15 for i in range(8)], -1).flatten(-2)


def per_value(c: torch.Tensor, dim: int) -> torch.Tensor:
    """Per-group constants [..., groups] -> [..., dim], in 64 bits."""
    return c.double().repeat_interleave(dim // c.shape[-1], -1)


def rows_of(arrays, table_row, positions, page):
    """(codes, scales, biases) of K and of V at a sequence's positions, [heads, positions, dim] in 64 bits."""
    pos = torch.as_tensor(positions, dtype=torch.long, device=arrays[0].device)
    pg = table_row.long()[pos // page]
    out = []
    for j in (0, 3):
        p, s, b = (a[pg, :, pos % page].transpose(0, 1) for a in arrays[j: j + 3])
        c = codes(p).double()
        out.append((c, per_value(s, c.shape[-1]), per_value(b, c.shape[-1])))
    return out


def many_rows(q, hk, seqs):
    """Whether the tensor-core kernel takes the call (launch_attn's rule)."""
    mean = -(-q.shape[0] // seqs)
    rows = (mean + mean // 2 if seqs > 1 else mean) * (q.shape[1] // hk)
    return rows > {64: 512, 128: 32, 256: math.inf}[q.shape[2]]


def attention(arrays, page, q, table, lens, cu, scale, window=0, tree=None):
    """(o, lse, o's bound, lse's bound) in 64 bits; rows of no sequence are NaN.

    The bounds follow the kernel's arithmetic.  Scores: fp32 sums of terms q * s * code and b * sum q,
    at most 2^-19 of their absolute sum off (D <= 256 terms, products exact).  Probabilities then carry
    twice that in relative terms (their own and the sum's) plus 2^-20 for exp2 and the fp32 sums.
    P * s is rounded to fp16 (2^-11 of it, times |code - 8|); below 2^-14 of the fp16 range it is
    subnormal, where the error is 2^-25 in units in which the row's largest P * s is 2^-4 at least,
    so 2^-18 of the largest P * s for each such position.  The result is rounded once.

    The kernel for many rows rounds V to fp16 instead (2^-11 |v|; a subnormal one by 2^-25), and P: once for bf16
    (2^-11, below 2^-14 by 2^-25 where the row's largest P is 1 at least), in two terms for fp16 (2^-22,
    covered by the score's share; the same below 2^-14)."""
    many = many_rows(q, arrays[0].shape[1], len(lens))
    T, H, D = q.shape
    hk = arrays[0].shape[1]
    grp = H // hk
    o = torch.full((T, H, D), math.nan, dtype=torch.float64, device=q.device)
    lse = torch.full((T, H), math.nan, dtype=torch.float64, device=q.device)
    ob, lb = torch.zeros_like(o), torch.zeros_like(lse)
    for b in range(len(lens)):
        r0, r1, n = int(cu[b]), int(cu[b + 1]), int(lens[b])
        new = r1 - r0
        if new == 0:
            continue
        o[r0:r1], lse[r0:r1] = 0, -math.inf
        if n <= 0:
            continue
        (kc, ks, kb), (vc, vs, vb) = rows_of(arrays, table[b], range(n), page)
        for i in range(new):
            pos = n - new + i
            at = torch.arange(n, device=q.device)
            if tree is None:
                sees = at <= pos
                if window:
                    sees &= at > pos - window
            else:
                d = at - (n - new)
                sees = (d < 0) | ((d < 64) & ((int(tree[r0 + i]) >> d.clamp(0, 63)) & 1).bool())
            idx = sees.nonzero().flatten()
            if idx.numel() == 0:
                continue
            for h in range(hk):
                x = q[r0 + i, h * grp: (h + 1) * grp].double()
                kk = ks[h, idx] * kc[h, idx] + kb[h, idx]
                vv = vs[h, idx] * vc[h, idx] + vb[h, idx]
                s = x @ kk.T * scale
                size = x.abs() @ (ks[h, idx].abs() * kc[h, idx] + kb[h, idx].abs()).T * abs(scale)
                w = torch.softmax(s, -1)
                hs = slice(h * grp, (h + 1) * grp)
                o[r0 + i, hs] = w @ vv
                lse[r0 + i, hs] = torch.logsumexp(s, -1)
                dx = 2.0 ** -19 * size.amax(-1, keepdim=True)
                ps = w[..., None] * vs[h, idx]  # [grp, positions, dim]
                top = ps.amax(1)
                low = (ps < top[:, None] * 2.0 ** -10).sum(1)
                ob[r0 + i, hs] = (2 * dx + 2.0 ** -20) * (w @ (vs[h, idx] * vc[h, idx] + vb[h, idx].abs() + 8 * vs[h, idx])) \
                    + 2.0 ** -11 * (w @ (vs[h, idx] * (vc[h, idx] - 8).abs())) + low * 2.0 ** -18 * top
                if many:
                    av = vv.abs()
                    wv = w @ av
                    ob[r0 + i, hs] = (2 * dx + 2.0 ** -20) * wv + 2.0 ** -11 * wv * (2 + 2.0 ** -10 if q.dtype == torch.bfloat16 else 1) \
                        + 2.0 ** -25 + idx.numel() * 2.0 ** -25 * w.amax(-1, keepdim=True) * av.amax(0)
                lb[r0 + i, hs] = dx.flatten() + 2.0 ** -21 * lse[r0 + i, hs].abs() + 2.0 ** -20
    return o, lse, ob + SIXTEEN[q.dtype] * (o.abs() + ob), lb
