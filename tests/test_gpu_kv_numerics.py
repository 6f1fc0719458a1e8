"""The K/V cache operators over values far from one: tiny groups, groups of different scale, one position that
outweighs a hundred thousand others."""
import math

import pytest
import torch

import bit_quantized_gemm_qmm_b200 as q
import kv_reference as ref
from test_gpu_kv import BF, HF, check, filled_cache, gen, ints, page_tables

pytestmark = pytest.mark.gpu


def one_sequence(tokens, page, seed=1):
    """A table of one sequence over pages in random order, and the pages' count."""
    pages = -(-tokens // page)
    order = torch.randperm(pages, device="cuda", generator=gen(seed)).to(torch.int32)
    return order[None].contiguous(), pages


@pytest.mark.parametrize("dtype", [HF, BF])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("tokens", [65, 2400])  # one word a thread, two
def test_append_of_tiny_groups(dtype, group, tokens):
    """Groups whose scale is a subnormal fp16 number, or rounds to zero: the scale is then off by up to half of
    its last place, however small it is, and the last codes lie beyond 15 before they are clamped."""
    dim, hk, page = 128, 8, 64
    table, pages = one_sequence(tokens, page)
    c = q.KVCache.empty(pages, page, hk, dim, group)
    amp = torch.logspace(-8, -4, tokens, device="cuda")[torch.randperm(tokens, device="cuda", generator=gen(2))]
    k, v = (torch.randn((tokens, hk, dim), device="cuda", generator=gen(j)) * amp[:, None, None] for j in (3, 4))
    v = v.abs() * torch.where(v.abs() > amp[:, None, None], 3.0, 0.01)  # most near the bias, some far
    k[7] = 0.0
    for i in range(20):  # exactly i + 1 steps of 2^-24 wide, times 15
        k[8 + i, :, ::2] = 0.0
        k[8 + i, :, 1::2] = (15 * (i // 2) + 7 * (i % 2) + 1) * 2.0 ** -24
    k[40, :, 1:], k[40, :, 0] = 0.0, 36 * 2.0 ** -24
    k, v = k.to(dtype), v.to(dtype)
    q.kv_append(c, k, v, table, ints([tokens]), ints([0, tokens]))
    for j, x in ((0, k), (3, v)):
        for a, part in zip(c.arrays()[j: j + 3], q.quantize(x.reshape(-1, dim), 4, group)):
            got = a[table[0].long()].transpose(1, 2).flatten(0, 1)[:tokens]  # [tokens, heads, ...]
            want = part.view(tokens, hk, -1)
            if a.dtype == HF:
                got, want = got.contiguous().view(torch.int16), want.view(torch.int16)
            wrong = (got != want).any(-1)
            assert not wrong.any(), f"{int(wrong.sum())} of {wrong.numel()} rows differ from quantize()'s"
    assert q.device_errors() == 0


# dim, group, heads a kv head, new tokens: the warps' kernel with one to four columns of query rows, the tensor-core kernel
@pytest.mark.parametrize("dim,group,grp,new", [(128, 64, 4, 2), (128, 32, 8, 1), (128, 64, 4, 4), (128, 64, 4, 5), (128, 32, 4, 8),
                                               (64, 32, 4, 2), (256, 64, 4, 2), (256, 32, 4, 3), (128, 64, 4, 12)])
@pytest.mark.parametrize("ratio", [8, 14])
def test_attention_of_v_groups_of_different_scale(dim, group, grp, new, ratio):
    """V's first group 2^ratio times the others: those are as exact as if they stood alone.

    Off, for a value of a group: the scores' and the sums' share, 2^-11 of each P * s times |code - 8| (the
    tensor-core kernel: of each P |v|), the output's rounding; and where a P * s lies 2^24 below the row's
    largest over all groups, so that it is subnormal in fp16, 2^-35 of that largest one, times 8."""
    n, hk, page = 1500, 2, 64
    table, pages = one_sequence(n, page)
    c = q.KVCache.empty(pages, page, hk, dim, group)
    k = torch.randn((n, hk, dim), device="cuda", generator=gen(3)).half()
    v = torch.randn((n, hk, dim), device="cuda", generator=gen(4)) * 4
    v[..., group:] *= 2.0 ** -ratio
    x = torch.randn((new, hk * grp, dim), device="cuda", generator=gen(5)).half()
    cu = ints([0, new])
    q.kv_append(c, k, v.half(), table, ints([n]), ints([0, n]))
    o, lse = q.kv_attention(c, x, table, ints([n]), cu)
    want, wl, _, bl = ref.attention(c.arrays(), page, x, table, [n], [0, new], dim ** -0.5)
    assert ((lse.double() - wl).abs() <= bl).all()
    (kc, ks, kb), (vc, vs, vb) = ref.rows_of(c.arrays(), table[0], range(n), page)
    many = ref.many_rows(x, hk, 1)
    for i in range(new):
        m = n - new + i + 1
        for h in range(hk):
            hs = slice(h * grp, (h + 1) * grp)
            xq = x[i, hs].double()
            w = torch.softmax(xq @ (ks * kc + kb)[h, :m].T * dim ** -0.5, -1)
            size = xq.abs() @ (ks * kc + kb.abs())[h, :m].T * dim ** -0.5
            dx = 2.0 ** -19 * size.amax(-1, keepdim=True)
            s, code, b = vs[h, :m], vc[h, :m], vb[h, :m].abs()
            bound = (2 * dx + 2.0 ** -19) * (w @ (s * code + b + 8 * s))
            if many:
                bound = bound + 2.0 ** -11 * (w @ (s * code + vb[h, :m]).abs()) + 2.0 ** -25
            else:
                ps = w[..., None] * s
                top = ps.amax((1, 2), keepdim=True)
                bound = bound + 2.0 ** -11 * (w @ (s * (code - 8).abs())) + ((ps < top * 2.0 ** -24).sum(1) * 2.0 ** -32) * top[:, 0]
            bound = bound + 2.0 ** -11 * (want[i, hs].abs() + bound) + 2.0 ** -25
            err = (o[i, hs].double() - want[i, hs]).abs()
            assert (err <= bound).all(), f"{(err / bound).max():.3g} of the bound, {(err / bound)[:, group:].max():.3g} past the first group"


@pytest.mark.parametrize("seqs,grp", [(1, 1), (600, 1), (1, 4), (1, 40), (300, 40)])
def test_attention_beside_one_large_weight(seqs, grp):
    """A first position whose weight is 2^21.2 times that of each of the 99,999 others (2^23.4 in the tensor-core
    kernel; they hold 4%, 0.9% together), read by many blocks and by one: the others count with what they hold.

    Off: the fp16 roundings of P * s (2^-11, times |code - 8|) or of V (2^-11 |v|), sums of fp32 that the matrix
    units truncate (2^-23 of the sum each step; a warp takes every fourth unit of 32 positions, two steps a unit;
    the tensor-core kernel every step of 16 itself), the scores' share (2^-19 of their size), the output's rounding."""
    n, dim, group, page = 100000, 128, 64, 1024
    table, pages = one_sequence(n, page)
    c = q.KVCache.empty(pages, page, 1, dim, group)
    for a, j in ((c.k_packed, 1), (c.v_packed, 2)):
        a.copy_(torch.randint(-2 ** 31, 2 ** 31 - 1, a.shape, device="cuda", generator=gen(j)))
    c.v_packed.bitwise_or_(-0x33333334)  # codes 12 to 15
    c.v_scales.fill_(0.1), c.v_biases.fill_(0.5)  # K is zero, but for
    x = torch.ones((seqs, grp, dim), device="cuda", dtype=HF)
    many = ref.many_rows(x, 1, seqs)
    c.k_biases[int(table[0, 0]), 0, 0] = (23.42 if many else 21.2) * math.log(2) / dim ** 0.5
    o, lse = q.kv_attention(c, x, table.expand(seqs, pages).contiguous(), ints([n] * seqs), ints(list(range(seqs + 1))))
    (kc, ks, kb), (vc, vs, vb) = ref.rows_of(c.arrays(), table[0], range(n), page)
    score = (ks * kc + kb)[0].sum(-1) * dim ** -0.5
    w = torch.softmax(score, -1)
    want, terms = w @ (vs * vc + vb)[0], w @ (vs * (vc + 8) + vb)[0]
    # a thread adds every 64th position or pair of positions (every 128th) to its sum, rounded by 2^-24 each time
    assert ((lse.double() - torch.logsumexp(score, -1)).abs() <= 2.0 ** -19 * score[0] + 2.0 ** -20 + n / 64 * 2.0 ** -24).all()
    steps = n / 16 if many else n / 64
    bound = 2.0 ** -11 * (want.abs() if many else w @ (vs * (vc - 8).abs())[0]) + (steps * 2.0 ** -23 + 2.0 ** -18 * score[0]) * terms
    bound = bound + 2.0 ** -11 * (want + bound)
    err = (o.double() - want).abs()
    assert (err <= bound).all(), f"off by {err.max():.3g}, {(err / bound).max():.3g} of the bound"


def poke(c, table, pos, group, **constants):
    """Sets a position's constants of one group of V (of all heads); its codes become 15."""
    pg, r = int(table[pos // c.page_size]), pos % c.page_size
    c.v_packed[pg, :, r] = -1
    for name, value in constants.items():
        getattr(c, name)[pg, :, r, group] = value


@pytest.mark.parametrize("dim,group,grp,new", [(128, 64, 4, 2), (128, 32, 4, 6), (64, 64, 4, 2), (256, 64, 4, 3), (128, 64, 4, 20),
                                             (128, 64, 4, 100), (128, 32, 4, 33), (64, 32, 16, 60), (128, 128, 8, 50)])
@pytest.mark.parametrize("name,value", [("v_scales", math.inf), ("v_scales", math.nan), ("v_biases", -math.inf), ("v_biases", math.nan)])
@pytest.mark.parametrize("at", [3, 697])
def test_attention_of_v_that_is_not_finite(dim, group, grp, new, name, value, at):
    """A position of the last group of V that holds an infinity or NaN: the lse knows nothing of it, nor do
    the other groups, nor the rows that do not see it."""
    n, hk, page = 700, 2, 64
    c = filled_cache(12, page, hk, dim, group, 1)
    table = page_tables([n], page, 12, 2)
    x = torch.randn((new, hk * grp, dim), device="cuda", generator=gen(5)).to(BF)
    lens, cu = ints([n]), ints([0, new])
    want, wl, bo, bl = ref.attention(c.arrays(), page, x, table, [n], [0, new], dim ** -0.5)
    poke(c, table[0], at, -1, **{name: value})
    if group < dim:  # its codes are others now
        keep = ref.attention(c.arrays(), page, x, table, [n], [0, new], dim ** -0.5)
        want[..., :-group], bo[..., :-group] = keep[0][..., :-group], keep[2][..., :-group]
    o, lse = q.kv_attention(c, x, table, lens, cu)
    assert ((lse.double() - wl).abs() <= bl).all()
    sees = torch.arange(new, device="cuda") + n - new >= at
    assert not o[sees][..., -group:].isfinite().any()
    ok = torch.ones_like(o, dtype=torch.bool)
    ok[sees, :, -group:] = False
    err = (o.double() - want).abs()
    assert (err[ok] <= bo[ok]).all(), f"off by {err[ok].max():.3g}"


@pytest.mark.parametrize("dim,group,grp,new,dtype", [(128, 64, 4, 20, HF), (128, 64, 4, 20, BF), (128, 64, 4, 100, BF), (128, 32, 4, 20, HF),
                                                     (128, 128, 8, 9, BF), (64, 32, 16, 60, HF), (64, 64, 16, 60, BF), (128, 64, 4, 2, HF)])
@pytest.mark.parametrize("mask", ["causal", "tree", "window", "seen by all"])
def test_attention_of_v_beyond_fp16(dim, group, grp, new, dtype, mask):
    """V whose finite constants give values past 65504 (60000 + 15 * 400): nothing to the rows that do not see it,
    itself to those that do."""
    n, hk, page = 700, 2, 64
    c = filled_cache(12, page, hk, dim, group, 1)
    table = page_tables([n], page, 12, 2)
    x = torch.randn((new, hk * grp, dim), device="cuda", generator=gen(5)).to(dtype)
    window, tree = 0, None
    if mask == "causal":
        at = [n - 1, n - new // 2]
    elif mask == "tree":
        at = [n - new + 1]
        tree = torch.randint(-2 ** 62, 2 ** 62, (new,), device="cuda", generator=gen(6)) | 1
    elif mask == "window":
        at, window = [n - 100 - new // 2, 100], 100
    else:
        at = [5, 300]
    for p in at:
        poke(c, table[0], p, -1, v_scales=400.0, v_biases=60000.0)
    lens, cu = ints([n]), ints([0, new])
    o, lse = q.kv_attention(c, x, table, lens, cu, window=window, tree=tree)
    want = ref.attention(c.arrays(), page, x, table, [n], [0, new], dim ** -0.5, window, tree)
    assert want[0].abs().max() < 65504  # of the output's range
    check(o, lse, want, mask)
    assert q.device_errors() == 0


# dim, group, heads a kv head, window, dtype, lens, new
@pytest.mark.parametrize("dim,group,grp,window,dtype,lens,new", [
    (128, 64, 3, 0, HF, [1, 2, 3, 2, 1, 2, 1], [1] * 7), (256, 64, 7, 0, HF, [1, 2] * 8, [1] * 16), (64, 64, 16, 3, HF, [1, 2, 4, 3], [1] * 4),
    (128, 128, 2, 1, HF, [500, 700], [3, 5]), (64, 32, 3, 2, HF, [100, 17, 64, 65], [2] * 4), (256, 32, 4, 2, BF, [300], [40]),
    (128, 128, 8, 1, HF, [600], [600]), (128, 64, 4, 2, HF, [300, 40], [300, 40]), (64, 32, 16, 1, HF, [200], [200]), (128, 32, 4, 1, HF, [90], [60]),
    (128, 64, 4, 1, BF, [600], [600]), (128, 64, 4, 2, BF, [90], [20])])
def test_lse_of_rows_that_see_one_or_two_positions(dim, group, grp, window, dtype, lens, new):
    """Their lse is the score of a position or two, with nothing to average: as a whole within 2^-21, some eight
    roundings of fp32 (dot products of up to 256 terms, s q code and b sum(q) several times their sum)."""
    hk, page = 2, 64
    need = sum(-(-n // page) for n in lens)
    c = filled_cache(need, page, hk, dim, group, 7, loud=1.0)
    table = page_tables(lens, page, need, 8)
    x = torch.randn((sum(new), hk * grp, dim), device="cuda", generator=gen(9)).to(dtype)
    cu = ints([sum(new[:i]) for i in range(len(new) + 1)])
    _, lse = q.kv_attention(c, x, table, ints(lens), cu, window=window)
    want = ref.attention(c.arrays(), page, x, table, lens, cu.tolist(), dim ** -0.5, window)[1]
    off = ((lse.double() - want).norm() / want.norm()).item()
    assert off <= 2.0 ** -21, f"{off:.3g}"


@pytest.mark.parametrize("dim,group,dtype", [(128, 64, BF), (128, 32, HF), (128, 128, BF), (64, 64, BF)])
def test_attention_of_decodes_beside_a_chunk(dim, group, dtype):
    """One long chunk of a prompt makes every sequence of the call many rows' kernel's: single tokens over caches of
    one position to a thousand, one without new tokens, a short draft."""
    hk, grp, page = 2, 8 if dim == 128 else 32, 64
    lens, new = [700, 1, 2, 128, 129, 1000, 300, 64, 37], [300, 1, 1, 1, 1, 1, 0, 1, 5]
    need = sum(-(-n // page) for n in lens)
    c = filled_cache(need, page, hk, dim, group, 11)
    table = page_tables(lens, page, need, 12)
    x = torch.randn((sum(new), hk * grp, dim), device="cuda", generator=gen(13)).to(dtype)
    assert ref.many_rows(x, hk, len(lens))
    cu = ints([sum(new[:i]) for i in range(len(new) + 1)])
    for window in (0, 50):
        o, lse = q.kv_attention(c, x, table, ints(lens), cu, window=window)
        check(o, lse, ref.attention(c.arrays(), page, x, table, lens, cu.tolist(), dim ** -0.5, window), f"window {window}")
    assert q.device_errors() == 0
