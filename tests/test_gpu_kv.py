"""The paged 4-bit K/V cache on a GPU: each operator against a plain 64-bit statement, at the sizes,
layouts and masks where it can go wrong."""
import math

import pytest
import torch

import bit_quantized_gemm_qmm_b200 as q
import kv_reference as ref

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def offsets(new):
    return ints([sum(new[:i]) for i in range(len(new) + 1)])


def filled_cache(pages, page, heads, dim, group, seed, loud=3.0):
    """A cache of quantized normal rows, a few K channels louder, through the library's own quantize()."""
    c = q.KVCache.empty(pages, page, heads, dim, group)
    for j, mul in ((0, loud), (3, 1.0)):
        x = torch.randn((pages * heads * page, dim), device="cuda", generator=gen(seed + j))
        x[:, :: max(1, dim // 5)] *= mul
        for a, part in zip(c.arrays()[j: j + 3], q.quantize(x.half(), 4, group)):
            a.copy_(part.view(a.shape))
    return c


def page_tables(lens, page, pages, seed, extra=0):
    """Tables of different pages in random order, -1 past each sequence's need."""
    need = [max(0, -(-n // page)) for n in lens]
    order = torch.randperm(pages, generator=gen(seed), device="cuda").to(torch.int32)
    assert sum(need) <= pages
    table = torch.full((len(lens), max(need + [1]) + extra), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at: at + n]
        at += n
    return table


def poison_unused(c, table, lens):
    """NaN constants in every row that no sequence's length covers."""
    used = torch.zeros(c.pages, c.page_size, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        for i in range(-(-n // c.page_size) if n > 0 else 0):
            used[int(table[b, i]), : min(c.page_size, n - i * c.page_size)] = True
    for a in (c.k_scales, c.k_biases, c.v_scales, c.v_biases):
        a[(~used)[:, None, :].expand(a.shape[:3])] = math.nan


def check(o, lse, want, what=""):
    wo, wl, bo, bl = want
    some = ~torch.isnan(wl)
    assert torch.equal(torch.isinf(lse[some]), torch.isinf(wl[some])), what
    fin = some & torch.isfinite(wl)
    err = (lse.double() - wl).abs()[fin]
    assert (err <= bl[fin]).all(), f"{what}: lse off by {err.max():.3g}, {(err / bl[fin]).max():.3g} of its bound"
    err = (o.double() - wo).abs()[some]
    ratio = (err / bo[some].clamp(min=1e-300)).nan_to_num(nan=0.0, posinf=math.inf)
    ok = err <= bo[some]
    assert ok.all(), f"{what}: o off by {err.max():.3g}, {ratio.max():.3g} of its bound, {int((~ok).sum())} values"


# name: dim, group, page, kv_heads, heads a kv head, dtype, lens, new, window, tree
ATTENTION = {
    "one token": (128, 64, 64, 8, 4, BF, [1024], [1], 0, False),
    "length one": (128, 64, 64, 2, 4, BF, [1], [1], 0, False),
    "ragged decodes": (128, 64, 64, 2, 4, BF, [1, 63, 64, 65, 300, 1999, 16, 17], [1] * 8, 0, False),
    "dim 64 group 32 page 16": (64, 32, 16, 3, 1, HF, [5, 100, 517], [1, 2, 3], 0, False),
    "dim 64 group 64": (64, 64, 32, 1, 8, HF, [5, 100, 517], [1, 1, 1], 0, False),
    "dim 64 wide": (64, 32, 128, 2, 16, BF, [257, 400], [3, 9], 0, False),
    "dim 128 group 32": (128, 32, 16, 2, 3, HF, [257, 40, 333], [4, 5, 1], 0, False),
    "dim 128 group 128": (128, 128, 256, 2, 5, BF, [257, 400], [2, 1], 0, False),
    "dim 128 group 32 wide": (128, 32, 16, 2, 7, HF, [257, 40, 333], [4, 5, 1], 0, False),
    "dim 256 group 32": (256, 32, 48, 1, 4, HF, [100, 401], [2, 1], 0, False),
    "dim 256 group 64 wide": (256, 64, 64, 2, 6, BF, [100, 401], [2, 5], 0, False),
    "dim 256 group 128": (256, 128, 64, 2, 2, HF, [100, 401], [2, 4], 0, False),
    "64 draft tokens": (128, 64, 64, 2, 4, BF, [300], [64], 0, False),
    "prompt": (128, 64, 64, 2, 2, HF, [333], [333], 0, False),
    "prompt chunks": (64, 64, 16, 1, 3, BF, [200, 131, 7], [77, 131, 0], 0, False),
    "no new tokens": (128, 64, 64, 2, 4, BF, [50, 90, 70], [0, 1, 0], 0, False),
    "shorter than its new tokens": (128, 64, 64, 2, 4, BF, [2, 0, 5], [5, 3, 5], 0, False),
    "window 1": (128, 64, 64, 2, 4, BF, [70, 200], [1, 3], 1, False),
    "window 50": (128, 64, 64, 2, 4, HF, [70, 200, 1000, 13], [1, 3, 1, 13], 50, False),
    "window over all": (128, 64, 64, 2, 4, HF, [70, 200], [1, 3], 5000, False),
    "window on a prompt": (64, 32, 16, 2, 2, BF, [400], [300], 33, False),
    "tree": (128, 64, 64, 2, 4, BF, [70, 200, 6, 64], [6, 5, 6, 1], 0, True),
    "tree of 64": (128, 32, 16, 2, 4, HF, [130, 64], [64, 64], 0, True),
    "mqa": (128, 64, 64, 1, 32, BF, [700, 33], [1, 2], 0, False),
    "mha": (128, 64, 64, 16, 1, HF, [260, 33], [1, 1], 0, False),
    "long": (128, 64, 64, 2, 4, HF, [20000], [2], 0, False),
    "long, one head": (64, 64, 64, 1, 1, BF, [100000], [1], 0, False),
    "long and short": (128, 64, 64, 1, 16, HF, [30000, 3, 40, 9000], [1, 1, 1, 1], 0, False),
    "32 rows": (128, 64, 64, 1, 4, BF, [900, 555], [8, 3], 0, False),
    "24 rows dim 64": (64, 32, 32, 2, 4, HF, [900, 31], [6, 2], 0, False),
    "33 rows": (128, 64, 64, 2, 33, BF, [700], [1], 0, False),
    "many rows dim 128 group 128": (128, 128, 64, 2, 4, BF, [700, 129], [40, 70], 0, False),
    "many rows dim 64 group 64": (64, 64, 16, 2, 8, BF, [257, 40], [40, 40], 0, False),
    "many rows dim 64 group 32 fp16": (64, 32, 48, 2, 5, HF, [1000], [50], 0, False),
    "many rows dim 128 group 128 fp16": (128, 128, 16, 1, 12, HF, [500, 77], [12, 30], 0, False),
    "many rows dim 128 group 32": (128, 32, 64, 1, 8, BF, [640], [20], 0, False),
    "prompt dim 64 group 64": (64, 64, 64, 1, 4, BF, [700], [200], 0, False),
    "prompt dim 64 group 32": (64, 32, 16, 1, 6, BF, [300], [150], 0, False),
    "prompt dim 64 fp16": (64, 32, 32, 1, 8, HF, [260, 131], [90, 40], 0, False),
    "prompt dim 128 group 128": (128, 128, 32, 1, 4, BF, [500], [129], 0, False),
    "many rows long": (128, 64, 64, 1, 8, BF, [40000], [9], 0, False),
    "many rows, some empty": (128, 64, 64, 2, 4, BF, [0, 300, 10, 64], [20, 0, 30, 64], 0, False),
    "many rows window 200": (128, 64, 64, 2, 4, BF, [1500, 130], [100, 130], 200, False),
    "many rows tree": (128, 64, 64, 2, 4, BF, [400, 40], [64, 33], 0, True),
    "dim 256 many rows": (256, 64, 16, 1, 8, BF, [300], [20], 0, False),
    "many short": (64, 64, 16, 2, 2, BF, [1 + (7 * i) % 23 for i in range(97)], [1] * 97, 0, False),
}


def attention_case(name, seed=1):
    dim, group, page, hk, grp, dtype, lens, new, window, tree = ATTENTION[name]
    need = sum(max(0, -(-n // page)) for n in lens)
    c = filled_cache(need + 2, page, hk, dim, group, seed)
    table = page_tables(lens, page, need + 2, seed + 10, extra=1)
    poison_unused(c, table, lens)
    T = sum(new)
    x = torch.randn((T, hk * grp, dim), device="cuda", generator=gen(seed + 20)).to(dtype)
    bits = None
    if tree:
        bits = torch.randint(-2 ** 63, 2 ** 63 - 1, (T,), device="cuda", generator=gen(seed + 30))
        bits[0] = 0  # sees the context only
    return c, x, table, ints(lens), offsets(new), dim ** -0.5, window, bits


@pytest.mark.parametrize("name", list(ATTENTION))
def test_attention(name):
    c, x, table, lens, cu, scale, window, bits = attention_case(name)
    o, lse = q.kv_attention(c, x, table, lens, cu, window=window, tree=bits)
    torch.cuda.synchronize()
    want = ref.attention(c.arrays(), c.page_size, x, table, lens.tolist(), cu.tolist(), scale, window, bits)
    check(o, lse, want, name)
    assert q.device_errors() == 0
    o2, lse2 = q.kv_attention(c, x, table, lens, cu, window=window, tree=bits)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)  # the order of sums is fixed


@pytest.mark.parametrize("name", ["one token", "ragged decodes", "dim 64 group 32 page 16", "dim 128 group 32 wide", "dim 256 group 32",
                                  "64 draft tokens", "many rows dim 64 group 32 fp16", "many rows dim 128 group 128"])
def test_attention_scores_are_fp32(name):
    """As a whole the lse is as near as a plain fp32 computation's (whose dot products of up to 256 terms and
    logarithm are some 2^-24 of their size off): a score that lost bits to 16-bit operands would be 2^-18 off."""
    c, x, table, lens, cu, scale, window, bits = attention_case(name)
    _, lse = q.kv_attention(c, x, table, lens, cu)
    want = ref.attention(c.arrays(), c.page_size, x, table, lens.tolist(), cu.tolist(), scale)[1]
    some = torch.isfinite(want)
    assert (lse.double() - want)[some].norm() <= 2.0 ** -21 * want[some].norm()


@pytest.mark.parametrize("dtype,amp,scale", [(BF, 2.0 ** 20, 1.0), (BF, 2.0 ** 60, 0.125), (BF, -(2.0 ** 24), 1.0), (BF, -(2.0 ** 103), 0.25),
                                             (HF, 60000.0, 1.0), (HF, 60000.0, 64.0), (HF, -60000.0, 8.0)])
@pytest.mark.parametrize("heads,new", [(4, 1), (4, 3), (8, 6)])
def test_attention_of_huge_scores(dtype, amp, scale, heads, new):
    """Scores far past 2^24, where the next fp32 number is many powers of e away: each row is V at the position of
    the largest score (others are 2^20 below it at least), and its lse that score.  Off by: V's or P * s's
    rounding to fp16 (2^-11, by the value or by 8 scales), fp32 sums (2^-18 of the terms), the output's rounding;
    the score by 2^-19 of its terms, all of one sign."""
    n, dim, group = 300, 128, 64
    c = filled_cache(8, 64, 2, dim, group, 31)
    k = 50 + torch.rand((c.pages * 2 * 64, dim), device="cuda", generator=gen(5)) * 4
    if amp > 0:
        k -= 49
    k = k.view(c.pages, 2, 64, dim)
    table = ints([[3, 1, 0, 5, 7]])
    best = 70  # of page 1
    k[1, :, best - 64] += 49 if amp > 0 else -49
    for a, part in zip(c.arrays()[:3], q.quantize(k.reshape(-1, dim).half(), 4, group)):
        a.copy_(part.view(a.shape))
    x = (amp * (0.5 + 0.5 * torch.rand((new, 2 * heads, dim), device="cuda", generator=gen(6)))).to(dtype)
    o, lse = q.kv_attention(c, x, table, ints([n]), ints([0, new]), scale=scale)
    (kc, ks, kb), (vc, vs, vb) = ref.rows_of(c.arrays(), table[0], [best], c.page_size)
    want = (x.double().view(new, 2, heads, dim) * (ks * kc + kb)[None]).sum(-1).view(new, -1) * scale
    assert ((lse.double() - want).abs() <= 2.0 ** -19 * want.abs()).all()
    v, s = ((vs * vc + vb)[:, 0], vs[:, 0].amax(-1, keepdim=True))
    bound = (2.0 ** -11 + 2.0 ** -14) * (8 * s + v.abs()) + 2.0 ** -18 * (16 * s + vb[:, 0].abs())
    bound = bound + ref.SIXTEEN[dtype] * (v.abs() + bound)
    err = (o.double().view(new, 2, heads, dim) - v[None, :, None]).abs()
    assert (err <= bound[None, :, None]).all(), (err / bound[None, :, None]).max()


def test_attention_strides_scale_and_outputs():
    """q as a slice of a fused projection's output at an odd offset, o and lse given, another scale."""
    c, x, table, lens, cu, _, _, _ = attention_case("ragged decodes")
    T, H, D = x.shape
    wide = torch.zeros((T, H * D + 17), dtype=x.dtype, device="cuda")
    view = wide[:, 3: 3 + H * D].unflatten(1, (H, D))
    view.copy_(x)
    out = torch.full((H, T + 2, D), 7.0, dtype=x.dtype, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    q.kv_attention(c, view, table, lens, cu, scale=0.25, out=out[:, 1: T + 1].transpose(0, 1), lse=lse)
    want = ref.attention(c.arrays(), c.page_size, x, table, lens.tolist(), cu.tolist(), 0.25)
    check(out[:, 1: T + 1].transpose(0, 1), lse, want)
    assert (out[:, 0] == 7).all() and (out[:, T + 1] == 7).all()


@pytest.mark.parametrize("name", ["many rows dim 128 group 128", "prompt dim 64 fp16", "32 rows"])
def test_attention_strides_other_kernels(name):
    c, x, table, lens, cu, scale, _, _ = attention_case(name)
    T, H, D = x.shape
    wide = torch.zeros((T, H * D + 17), dtype=x.dtype, device="cuda")
    view = wide[:, 3: 3 + H * D].unflatten(1, (H, D))
    view.copy_(x)
    out = torch.full((H, T + 2, D), 7.0, dtype=x.dtype, device="cuda")
    plain, lse = q.kv_attention(c, x, table, lens, cu)
    _, lse2 = q.kv_attention(c, view.requires_grad_(False), table, lens, cu, out=out[:, 1: T + 1].transpose(0, 1))
    assert torch.equal(out[:, 1: T + 1].transpose(0, 1), plain) and torch.equal(lse, lse2)
    assert (out[:, 0] == 7).all() and (out[:, T + 1] == 7).all()
    # without an lse, through the C ABI; and the call on a leaf that requires a gradient reads it as it is
    import ctypes
    o = torch.full_like(x, 7.0)
    s = q.SeqsDesc(table.data_ptr(), cu.data_ptr(), table.shape[0], table.stride(0), table.shape[1])
    st = q.lib().qmm_kv_attention(ctypes.byref(c._desc), x.data_ptr(), H * D, D, o.data_ptr(), H * D, D, None, ctypes.byref(s),
                                  lens.data_ptr(), T, H, scale, 0, None, q.QMM_BF16 if x.dtype == BF else q.QMM_F16,
                                  torch.cuda.current_stream().cuda_stream)
    assert st == q.QMM_OK and torch.equal(o, plain)
    leaf = x.detach().clone().requires_grad_(True)
    assert torch.equal(q.kv_attention(c, leaf, table, lens, cu)[0].detach(), plain)


@pytest.mark.parametrize("name", ["ragged decodes", "many rows dim 128 group 128"])
def test_attention_leaves_rows_of_no_sequence(name):
    c, x, table, lens, cu, scale, _, _ = attention_case(name)
    T, H, D = x.shape
    pad = torch.cat([x[:2], x, x[:3]])
    out, lse = torch.full((T + 5, H, D), 7.0, dtype=x.dtype, device="cuda"), torch.full((T + 5, H), 7.0, device="cuda")
    q.kv_attention(c, pad, table, lens, cu + 2, out=out, lse=lse)
    want = ref.attention(c.arrays(), c.page_size, x, table, lens.tolist(), cu.tolist(), scale)
    check(out[2: T + 2], lse[2: T + 2], want)
    for t in (out, lse):
        assert (t[:2] == 7).all() and (t[T + 2:] == 7).all()


@pytest.mark.parametrize("name", ["tree", "many rows tree", "tree of 64"])
def test_attention_does_not_see_nan_and_infinity_behind_the_mask(name):
    """Draft rows that a token's tree mask or position hides may hold anything."""
    c, x, table, lens, cu, scale, _, _ = attention_case(name)
    T = x.shape[0]
    bits = torch.ones(T, dtype=torch.int64, device="cuda")  # everyone sees draft token 0 of its sequence only
    want = ref.attention(c.arrays(), c.page_size, x, table, lens.tolist(), cu.tolist(), scale, 0, bits)
    for b, n in enumerate(lens.tolist()):
        new = int(cu[b + 1] - cu[b])
        for i in range(1, new):
            pos = n - new + i
            pg, r = int(table[b, pos // c.page_size]), pos % c.page_size
            for a, v in ((c.k_scales, math.nan), (c.k_biases, math.inf), (c.v_scales, math.inf), (c.v_biases, math.nan)):
                a[pg, :, r] = v
    check(*q.kv_attention(c, x, table, lens, cu, tree=bits), want)
    # causal: the first token of each sequence sees none of them, the others read as NaN
    o, lse = q.kv_attention(c, x, table, lens, cu)
    causal = ref.attention(c.arrays(), c.page_size, x, table, lens.tolist(), cu.tolist(), scale)
    first = cu[:-1].long()
    check(o[first], lse[first], [t[first] for t in causal])
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[first] = False
    assert o[rest].isnan().all()


def test_attention_nan_query_stays_in_its_row():
    c, x, table, lens, cu, scale, _, _ = attention_case("64 draft tokens")
    want = ref.attention(c.arrays(), c.page_size, x, table, lens.tolist(), cu.tolist(), scale)
    x = x.clone()
    x[5, 2, 7], x[6, 0, 0] = math.nan, math.inf
    o, lse = q.kv_attention(c, x, table, lens, cu)
    assert o[5, 2].isnan().all() and o[6, 0].isnan().all()
    o[5, 2], o[6, 0], lse[5, 2], lse[6, 0] = want[0][5, 2].to(o.dtype), want[0][6, 0].to(o.dtype), want[1][5, 2], want[1][6, 0]
    check(o, lse, want)


@pytest.mark.parametrize("new", [2, 40])
@pytest.mark.parametrize("what", ["large V", "small V", "V of one value", "zero V", "loud late key", "rising keys", "small q",
                                  "large q", "mixed V"])
def test_attention_ranges(what, new):
    """Values far from one: the running references must follow them (both kernels)."""
    dim, group, page, hk, grp = 128, 64, 64, 2, 4
    n, pages = 1500, 24
    c = q.KVCache.empty(pages, page, hk, dim, group)
    k = torch.randn((n, hk, dim), device="cuda", generator=gen(3))
    v = torch.randn((n, hk, dim), device="cuda", generator=gen(4))
    x = torch.randn((new, hk * grp, dim), device="cuda", generator=gen(5))
    if what == "large V":
        v = v * 12000
    if what == "small V":
        v = v * 2e-4
    if what == "V of one value":
        v = torch.full_like(v, 3.0)
    if what == "zero V":
        v = torch.zeros_like(v)
    if what == "mixed V":
        v = v * torch.logspace(-3, 3, n, device="cuda")[:, None, None]
    if what == "loud late key":
        k[1400] = 8 * x[0].view(hk, grp, dim)[:, 0]
    if what == "rising keys":
        k = k + x[1].view(hk, grp, dim)[:, 1] * torch.linspace(0, 6, n, device="cuda")[:, None, None]
    if what == "small q":
        x = x * 1e-4
    if what == "large q":
        x = x * 60
    x, k, v = x.half(), k.clamp(-6e4, 6e4).half(), v.clamp(-6e4, 6e4).half()
    table = page_tables([n], page, pages, 6)
    lens = ints([n])
    q.kv_append(c, k, v, table, lens, ints([0, n]))
    cu = ints([0, new])
    o, lse = q.kv_attention(c, x, table, lens, cu)
    want = ref.attention(c.arrays(), page, x, table, [n], [0, new], dim ** -0.5)
    check(o, lse, want, what)
    if what == "zero V":
        assert (o == 0).all()


def test_attention_bad_pages_many_rows():
    """The same in the kernel for many rows: what a missing page would have held is left out."""
    c, x, table, lens, cu, scale, _, _ = attention_case("many rows dim 128 group 128")
    for bad in (-1, c.pages, -2 ** 31):
        t2 = table.clone()
        t2[0, 3] = bad  # positions 192..255 of the sequence of 700
        o, lse = q.kv_attention(c, x, t2, lens, cu)
        torch.cuda.synchronize()
        assert q.device_errors() == 2
        keep = [p for p in range(700) if not 192 <= p < 256]
        (kc, ks, kb), (vc, vs, vb) = ref.rows_of(c.arrays(), table[0], keep, c.page_size)
        last = 39  # sees all of them
        s = torch.einsum("hd,htd->ht", x[last].double(), (ks * kc + kb).repeat_interleave(4, 0)) * scale
        assert torch.allclose(lse[last].double(), torch.logsumexp(s, -1), atol=1e-4)
        ok = ref.attention(c.arrays(), c.page_size, x, table, lens.tolist(), cu.tolist(), scale)
        check(o[40:], lse[40:], [t[40:] for t in ok])


def test_attention_bad_pages_and_lengths():
    """Pages outside the pool and positions outside the table are left out, and say so."""
    c, x, table, lens, cu, scale, _, _ = attention_case("ragged decodes")
    for bad in (-1, c.pages, 2 ** 31 - 1, -2 ** 31):
        t2 = table.clone()
        t2[5, 3] = bad  # positions 192..255 of the sequence of 1999
        o, lse = q.kv_attention(c, x, t2, lens, cu)
        torch.cuda.synchronize()
        assert q.device_errors() == 2
        keep = [p for p in range(1999) if not 192 <= p < 256]
        (kc, ks, kb), (vc, vs, vb) = ref.rows_of(c.arrays(), table[5], keep, c.page_size)
        s = torch.einsum("hd,htd->ht", x[5].double(), (ks * kc + kb).repeat_interleave(4, 0)) * scale
        assert torch.allclose(lse[5].double(), torch.logsumexp(s, -1), atol=1e-4)
        ok = ref.attention(c.arrays(), c.page_size, x, table, lens.tolist(), cu.tolist(), scale)
        rows = [b for b in range(8) if b != 5]
        check(o[rows], lse[rows], [t[rows] for t in ok])
    # a length past the table: what the table names is seen, the poisoned rows behind the first too
    longer = lens.clone()
    longer[0] = 10 ** 9
    o, lse = q.kv_attention(c, x, table[:, :1], longer, cu)
    torch.cuda.synchronize()
    assert q.device_errors() == 2 and lse[0].isnan().all()
    # offsets that leave the rows, and that fall (nothing is done)
    for off in ([-7, 1, 2, 3, 4, 5, 6, 7, 10 ** 6], [8] * 9, [0] * 9):
        q.kv_attention(c, x, table, lens, ints(off))
    torch.cuda.synchronize()
    q.device_errors()
    out = torch.full_like(x, 7.0)
    for off in ([0, 5, 2, 3, 4, 5, 6, 7, 8], [2 ** 31 - 1, -2 ** 31] * 4 + [0]):
        q.kv_attention(c, x, table, lens, ints(off), out=out)
        torch.cuda.synchronize()
        assert q.device_errors() == 2 and (out == 7).all()
    q.kv_attention(c, x, table, ints([-5, -2 ** 31, 0, 1, 2, 3, 4, 5]), cu)
    torch.cuda.synchronize()
    q.device_errors()


def test_attention_empty_calls():
    c = q.KVCache.empty(2, 16, 1, 64, 64)
    x = torch.zeros((0, 2, 64), dtype=HF, device="cuda")
    o, lse = q.kv_attention(c, x, ints([[0]]), ints([0]), ints([0, 0]))
    assert o.shape == (0, 2, 64) and lse.shape == (0, 2)
    x = torch.ones((3, 2, 64), dtype=HF, device="cuda")
    o, lse = q.kv_attention(c, x, torch.empty((1, 0), dtype=torch.int32, device="cuda"), ints([0]), ints([0, 3]))
    assert (o == 0).all() and (lse == -math.inf).all()
    out = torch.full_like(x, 5.0)
    q.kv_attention(c, x, torch.empty((0, 1), dtype=torch.int32, device="cuda"), ints([]), ints([0]), out=out)
    assert (out == 5).all()
    torch.cuda.synchronize()


# dim, group, page, kv_heads, dtype, lens, new
APPEND = [
    (128, 64, 64, 8, BF, [2000, 1, 64, 65], [1, 1, 1, 1]),
    (128, 64, 64, 2, HF, [333], [333]),
    (64, 32, 16, 1, HF, [1], [1]),
    (64, 64, 16, 3, BF, [17, 40, 9], [17, 0, 5]),
    (128, 32, 32, 5, BF, [70, 31], [33, 31]),
    (128, 128, 16, 1, HF, [40, 17], [9, 17]),
    (256, 64, 64, 2, HF, [100, 64, 63], [50, 3, 63]),
    (256, 128, 16, 1, BF, [100, 64, 63], [50, 3, 63]),
    (256, 32, 48, 4, BF, [7], [7]),
    (64, 64, 16, 2, HF, [3 + i % 40 for i in range(150)], [1 + i % 3 for i in range(150)]),
]


def append_case(dim, group, page, hk, dtype, lens, new, seed=2):
    need = sum(-(-n // page) for n in lens)
    c = filled_cache(need + 2, page, hk, dim, group, seed)
    table = page_tables(lens, page, need + 2, seed + 1)
    k, v = (torch.randn((sum(new), hk, dim), device="cuda", generator=gen(seed + j)).to(dtype) for j in (5, 6))
    return c, k, v, table, ints(lens), offsets(new)


def expected_append(c, k, v, table, lens, new):
    """The six arrays after an append, by quantize() of the rows and indexing."""
    want = [a.clone() for a in c.arrays()]
    r = 0
    for b, (n, m) in enumerate(zip(lens, new)):
        for i in range(m):
            pos = n - m + i
            pg, row = int(table[b, pos // c.page_size]), pos % c.page_size
            for j, x in ((0, k), (3, v)):
                for a, part in zip(want[j: j + 3], q.quantize(x[r + i].contiguous(), 4, c.group)):
                    a[pg, :, row] = part
        r += m
    return want


@pytest.mark.parametrize("case", APPEND)
def test_append_is_quantize_and_gather_dequantize(case):
    dim, group, page, hk, dtype, lens, new = case
    c, k, v, table, tl, cu = append_case(*case)
    k[0, 0, :group] = 2.5            # a group of one value
    v[-1, -1, group // 2:] = 0.0
    v[-1, -1, : group // 2] = -0.0   # zeros of both signs
    want = expected_append(c, k, v, table, lens, new)
    q.kv_append(c, k, v, table, tl, cu)
    torch.cuda.synchronize()
    for name, a, w in zip(("kp", "ks", "kb", "vp", "vs", "vb"), c.arrays(), want):
        assert torch.equal(a.view(torch.int16) if a.dtype == HF else a, w.view(torch.int16) if w.dtype == HF else w), name
    starts = ints([n - m for n, m in zip(lens, new)])
    for dt in (HF, BF):
        gk, gv = q.kv_gather(c, table, starts, cu, sum(new), dt)
        for x, got in ((k, gk), (v, gv)):
            p = q.quantize(x.reshape(-1, dim).contiguous(), 4, group)
            assert torch.equal(q.dequantize(*p, dim, 4, group, dtype=dt).view(got.shape), got)
    assert q.device_errors() == 0


def test_append_strided_and_unaligned_rows():
    case = APPEND[3]
    dim, group, page, hk, dtype, lens, new = case
    c, k, v, table, tl, cu = append_case(*case)
    want = expected_append(c, k, v, table, lens, new)
    T = sum(new)
    wide = torch.zeros((T, 2 * hk * dim + 5), dtype=dtype, device="cuda")  # a fused k/v projection at an odd offset
    kk = wide[:, 1: 1 + hk * dim].unflatten(1, (hk, dim))
    vv = wide[:, 1 + hk * dim: 1 + 2 * hk * dim].unflatten(1, (hk, dim))
    kk.copy_(k), vv.copy_(v)
    q.kv_append(c, kk, vv, table, tl, cu)
    assert all(torch.equal(a, w) for a, w in zip(c.arrays(), want))
    # heads first, on a fresh cache
    c2, *_ = append_case(*case)
    q.kv_append(c2, k.transpose(0, 1).contiguous().transpose(0, 1), v, table, tl, cu)
    assert all(torch.equal(a, w) for a, w in zip(c2.arrays(), want))


def test_append_and_gather_leave_the_rest():
    """Rows of no sequence are not read into the cache nor written by a gather."""
    case = APPEND[4]
    dim, group, page, hk, dtype, lens, new = case
    c, k, v, table, tl, cu = append_case(*case)
    want = expected_append(c, k, v, table, lens, new)
    T = sum(new)
    pad = lambda x: torch.cat([torch.full_like(x[:3], 9), x, torch.full_like(x[:2], 9)])  # noqa: E731
    q.kv_append(c, pad(k), pad(v), table, tl, cu + 3)
    assert all(torch.equal(a, w) for a, w in zip(c.arrays(), want))
    out = tuple(torch.full((hk, T + 5, dim), 7.0, dtype=dtype, device="cuda").transpose(0, 1) for _ in range(2))
    starts = ints([n - m for n, m in zip(lens, new)])
    q.kv_gather(c, table, starts, cu + 3, T + 5, dtype, out=out)
    plain = q.kv_gather(c, table, starts, cu, T, dtype)
    for o, p in zip(out, plain):
        assert torch.equal(o[3: T + 3], p) and (o[:3] == 7).all() and (o[T + 3:] == 7).all()


def test_append_not_finite_reads_as_nan():
    c, k, v, table, tl, cu = append_case(*APPEND[1])
    k, v = k.float(), v.float()
    k[3, 1, 70], v[4, 0, 3], v[5, 1, 100] = math.nan, math.inf, -math.inf
    k, v = k.bfloat16(), v.bfloat16()
    k[6, 0, 0], k[7, 0, 0] = 1e6, -1e6  # the scale, then the bias, beyond fp16
    q.kv_append(c, k, v, table, tl, cu)
    gk, gv = q.kv_gather(c, table, ints([0]), cu, 333)
    nk, nv = torch.zeros_like(gk, dtype=torch.bool), torch.zeros_like(gv, dtype=torch.bool)
    nk[3, 1, 64:], nv[4, 0, :64], nv[5, 1, 64:], nk[7, 0, :64] = True, True, True, True
    nk[6, 0, :64] = True  # 1e6 / 15 > 65504
    assert torch.equal(gk.isnan(), nk) and torch.equal(gv.isnan(), nv)


def test_append_gather_bad_pages():
    case = APPEND[1]
    dim, group, page, hk, dtype, lens, new = case
    c, k, v, table, tl, cu = append_case(*case)
    want = expected_append(c, k, v, table, lens, new)
    before = [a.clone() for a in c.arrays()]
    page2 = int(table[0, 2])
    t2 = table.clone()
    t2[0, 2] = c.pages
    q.kv_append(c, k, v, t2, tl, cu)
    torch.cuda.synchronize()
    assert q.device_errors() == 2
    for a, w, old in zip(c.arrays(), want, before):
        w[page2] = old[page2]
        assert torch.equal(a, w)
    gk, gv = q.kv_gather(c, t2, ints([0]), cu, 333)
    torch.cuda.synchronize()
    assert q.device_errors() == 2
    assert (gk[128:192] == 0).all() and (gv[128:192] == 0).all() and not (gk[:128] == 0).all()
    q.kv_gather(c, table, ints([-5]), cu, 333)       # positions in front of the sequence
    q.kv_append(c, k, v, table, ints([300]), cu)     # a length below its new tokens
    torch.cuda.synchronize()
    assert q.device_errors() == 2


# dim, group, page, kv_heads, pages, pairs
@pytest.mark.parametrize("dim,group,page,hk,pages,pairs", [
    (128, 64, 64, 8, 40, 17), (64, 64, 16, 1, 9, 1), (64, 32, 16, 3, 700, 333), (256, 32, 256, 8, 8, 3),
    (256, 128, 48, 2, 30, 15), (128, 128, 1024, 1, 4, 2)])
def test_copy_pages(dim, group, page, hk, pages, pairs):
    c = filled_cache(pages, page, hk, dim, group, 3)
    order = torch.randperm(pages, device="cuda", generator=gen(4)).to(torch.int32)
    src, dst = order[:pairs].clone(), order[pairs: 2 * pairs].clone()
    if pairs > 2:
        src[2] = src[0]  # one page to two places
    want = [a.clone() for a in c.arrays()]
    for w, a in zip(want, c.arrays()):
        w[dst.long()] = a[src.long()]
    q.kv_copy_pages(c, src, dst)
    torch.cuda.synchronize()
    assert all(torch.equal(a, w) for a, w in zip(c.arrays(), want))
    assert q.device_errors() == 0


def test_copy_pages_same_target_and_refusals():
    c = filled_cache(12, 16, 2, 64, 32, 3)
    old = [a.clone() for a in c.arrays()]
    # target 5 twice: the last counts; 7 -> 7 is nothing; 1 -> 2 -> 3 would be torn: 2 -> 3 is skipped
    q.kv_copy_pages(c, ints([0, 4, 7, 1, 2]), ints([5, 5, 7, 2, 3]))
    torch.cuda.synchronize()
    assert q.device_errors() == 2
    for a, o in zip(c.arrays(), old):
        w = o.clone()
        w[5], w[2] = o[4], o[1]
        assert torch.equal(a, w)
    q.kv_copy_pages(c, ints([0, 12, -1, 3]), ints([-1, 1, 1, 2 ** 31 - 1]))
    torch.cuda.synchronize()
    assert q.device_errors() == 2
    q.kv_copy_pages(c, ints([]), ints([]))


# dim, group, page, kv_heads, starts, keep
COMPACT = [
    (128, 64, 64, 8, [1024], [[0, 2, 5]]),
    (64, 32, 16, 1, [0, 15, 31], [[1], [0, 1, 2], [3, 4, 5, 6, 40]]),
    (256, 32, 16, 3, [10, 5], [[], list(range(1, 64, 2))]),
    (256, 128, 64, 2, [62, 100], [list(range(64)), list(range(1, 65))]),
    (128, 128, 32, 2, [3], [[i + i // 3 for i in range(150)]]),
]


@pytest.mark.parametrize("dim,group,page,hk,starts,keep", COMPACT)
def test_compact(dim, group, page, hk, starts, keep):
    lens = [s + (max(k) + 1 if k else 1) for s, k in zip(starts, keep)]
    need = sum(-(-n // page) for n in lens)
    c = filled_cache(need + 1, page, hk, dim, group, 8)
    table = page_tables(lens, page, need + 1, 9)
    want = [a.clone() for a in c.arrays()]
    for b, (s, mine) in enumerate(zip(starts, keep)):
        for w, a in zip(want, c.arrays()):
            for j, m in enumerate(mine):
                to, fr = s + j, s + m
                w[int(table[b, to // page]), :, to % page] = a[int(table[b, fr // page]), :, fr % page]
    flat = [m for mine in keep for m in mine]
    q.kv_compact(c, table, ints(starts), ints(flat), offsets([len(k) for k in keep]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, w) for a, w in zip(c.arrays(), want))
    assert q.device_errors() == 0


def test_compact_bad_positions():
    c = filled_cache(4, 16, 2, 64, 64, 8)
    old = [a.clone() for a in c.arrays()]
    table = ints([[0, 1], [2, -1]])
    # beyond the table, a missing page, in front of the sequence
    q.kv_compact(c, table, ints([20, 10]), ints([30, 8, -3]), ints([0, 1, 3]))
    torch.cuda.synchronize()
    assert q.device_errors() == 2
    assert all(torch.equal(a, o) for a, o in zip(c.arrays(), old))
    q.kv_compact(c, table, ints([-4, 10 ** 9]), ints([0, 1]), ints([-5, 1, 10 ** 6]))
    torch.cuda.synchronize()
    assert q.device_errors() == 2


def test_rows_beyond_32_bits():
    """A cache whose arrays pass 2^32 bytes: pages at both ends."""
    pages, page, hk, dim, group = 35000, 64, 16, 128, 64
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GB")
    c = q.KVCache.empty(pages, page, hk, dim, group)
    assert c.k_packed.numel() * 4 > 2 ** 31
    lens, new = [100, 70], [100, 70]
    table = ints([[pages - 1, 0], [pages - 2, 17]])
    k, v = (torch.randn((170, hk, dim), device="cuda", generator=gen(j)).to(BF) for j in (5, 6))
    q.kv_append(c, k, v, table, ints(lens), offsets(new))
    small = q.KVCache.empty(4, page, hk, dim, group)
    at = ints([[3, 0], [2, 1]])
    q.kv_append(small, k, v, at, ints(lens), offsets(new))
    for a, s in zip(c.arrays(), small.arrays()):
        assert torch.equal(a[[0, 17, pages - 2, pages - 1]], s)
    x = torch.randn((2, 32, dim), device="cuda", generator=gen(7)).to(BF)
    o, lse = q.kv_attention(c, x, table, ints(lens), ints([0, 1, 2]))
    o2, lse2 = q.kv_attention(small, x, at, ints(lens), ints([0, 1, 2]))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    q.kv_copy_pages(c, ints([pages - 1]), ints([pages - 3]))
    for a in c.arrays():
        assert torch.equal(a[pages - 3], a[pages - 1])


def test_streams_and_graphs():
    """Calls on a side stream, and a captured decode step replayed with other lengths, pages and values;
    two graphs that overlap keep apart."""
    dim, group, page, hk, grp = 128, 64, 64, 4, 4
    graphs = []
    for s in range(2):
        lens, new = [300 + s, 900, 64], [1, 1, 1]
        c, k, v, table, tl, cu = append_case(dim, group, page, hk, BF, lens, new, seed=20 + s)
        x = torch.randn((3, hk * grp, dim), device="cuda", generator=gen(30 + s)).to(BF)
        out, lse = torch.empty_like(x), torch.empty((3, hk * grp), device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            q.kv_append(c, k, v, table, tl, cu)
            q.kv_attention(c, x, table, tl, cu, out=out, lse=lse)
        torch.cuda.current_stream().wait_stream(side)
        check(out, lse, ref.attention(c.arrays(), page, x, table, lens, cu.tolist(), dim ** -0.5))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q.kv_append(c, k, v, table, tl, cu)
            q.kv_attention(c, x, table, tl, cu, out=out, lse=lse)
        graphs.append((g, c, k, v, table, tl, cu, x, out, lse))
    streams = [torch.cuda.Stream() for _ in graphs]
    for turn in range(3):
        for s, (g, c, k, v, table, tl, cu, x, out, lse) in enumerate(graphs):
            tl.copy_(ints([200 + 7 * turn, 900 - 300 * turn, 1 + turn]))
            table.copy_(table.roll(1, 0) if turn == 1 else table)
            if turn == 1:
                table.clamp_(min=0)
            x.copy_(torch.randn(x.shape, device="cuda", generator=gen(50 + turn)))
            k.copy_(torch.randn(k.shape, device="cuda", generator=gen(60 + turn)))
        torch.cuda.synchronize()
        for _ in range(5):
            for st, (g, *_rest) in zip(streams, graphs):
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        for g, c, k, v, table, tl, cu, x, out, lse in graphs:
            check(out, lse, ref.attention(c.arrays(), page, x, table, tl.tolist(), cu.tolist(), dim ** -0.5), f"turn {turn}")
    q.device_errors()


def test_python_refusals():
    c = q.KVCache.empty(4, 16, 2, 64, 64)
    x = torch.zeros((2, 4, 64), dtype=HF, device="cuda")
    k = torch.zeros((2, 2, 64), dtype=HF, device="cuda")
    table, lens, cu = ints([[0, 1]]), ints([5]), ints([0, 2])
    bad = [
        lambda: q.kv_attention(c, x[:, :3], table, lens, cu),
        lambda: q.kv_attention(c, x[..., :32], table, lens, cu),
        lambda: q.kv_attention(c, x.float(), table, lens, cu),
        lambda: q.kv_attention(c, x.cpu(), table, lens, cu),
        lambda: q.kv_attention(c, x, table.long(), lens, cu),
        lambda: q.kv_attention(c, x, table[0], lens, cu),
        lambda: q.kv_attention(c, x, table, lens.long(), cu),
        lambda: q.kv_attention(c, x, table, lens, cu[:1]),
        lambda: q.kv_attention(c, x, table, lens, cu, window=-1),
        lambda: q.kv_attention(c, x, table, lens, cu, tree=lens),
        lambda: q.kv_attention(c, x, table, lens, cu, window=3, tree=torch.zeros(2, dtype=torch.int64, device="cuda")),
        lambda: q.kv_attention(c, x, table, lens, cu, out=x[:1]),
        lambda: q.kv_attention(c, x, table, lens, cu, lse=torch.zeros((2, 3), device="cuda")),
        lambda: q.kv_append(c, k, x, table, lens, cu),
        lambda: q.kv_append(c, k, k.bfloat16(), table, lens, cu),
        lambda: q.kv_append(c, k, k[:1], table, lens, cu),
        lambda: q.kv_gather(c, table, lens, cu, 3, HF, out=(k, k)),
        lambda: q.kv_gather(c, table, lens, cu, 2, BF, out=(k, k)),
        lambda: q.kv_copy_pages(c, lens, cu),
        lambda: q.kv_compact(c, table, lens, cu.long(), cu),
        lambda: q.KVCache(*[a[:, :, ::2] for a in c.arrays()], group=64),
        lambda: q.KVCache(*c.arrays(), group=32),
        lambda: q.KVCache.empty(4, 16, 2, 64, 48),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, q.QmmError)):
            f()
            pytest.fail(f"case {i} was taken")
    for kw in (dict(page_size=8), dict(page_size=24), dict(head_dim=96, group=32), dict(page_size=2048)):
        a = dict(pages=2, page_size=16, kv_heads=1, head_dim=64, group=64)
        a.update(kw)
        c2 = q.KVCache.empty(**a)
        with pytest.raises(q.QmmError):
            q.kv_copy_pages(c2, ints([0]), ints([1]))


def test_sequences_together():
    """A serving loop: prompts, forks, draft trees verified and accepted, ends; every step's attention
    against the same tokens kept as plain rows."""
    dim, group, page, hk, grp = 64, 32, 16, 2, 3
    c = q.KVCache.empty(60, page, hk, dim, group)
    s = q.KVSequences(c)
    rows = {}  # sequence -> list of (k, v) rows as the cache keeps them
    g = gen(77)

    def back(x):
        p = q.quantize(x.reshape(-1, dim).contiguous(), 4, group)
        return q.dequantize(*p, dim, 4, group, dtype=HF).view(x.shape)

    def step(seqs, new, tree=None):
        n = sum(new)
        x = torch.randn((n, hk * grp, dim), device="cuda", generator=g).half()
        k, v = (torch.randn((n, hk, dim), device="cuda", generator=g).half() for _ in range(2))
        o = s.step(seqs, x, k, v, new, tree=tree)
        r = 0
        for name, m in zip(seqs, new):
            rows[name] = rows[name] + list(zip(back(k[r: r + m]), back(v[r: r + m])))
            assert s.length(name) == len(rows[name])
            kk, vv = (torch.stack([p[i] for p in rows[name]]).double() for i in (0, 1))
            for i in range(m):
                at = torch.arange(len(rows[name]), device="cuda")
                first = len(rows[name]) - m
                sees = at <= first + i if tree is None else \
                    (at < first) | ((int(tree[r + i]) >> (at - first).clamp(0, 63)) & 1).bool()
                w = torch.softmax(torch.einsum("hgd,thd->hgt", x[r + i].double().view(hk, grp, dim), kk[sees]) * dim ** -0.5, -1)
                want = torch.einsum("hgt,thd->hgd", w, vv[sees]).reshape(hk * grp, dim)
                # |v| <= 6: fp16 rounding of P*s, of the rows read back and of the result, 2^-11 each, against rows of size <= 6
                assert (o[r + i].double() - want).abs().max() <= 3 * 2.0 ** -11 * 6
            r += m

    a = s.add()
    rows[a] = []
    step([a], [37])
    b = s.fork(a)
    rows[b] = list(rows[a])
    step([a, b], [1, 1])
    tree = torch.tensor([1, 3, 5, 11, 1, 3, 7], dtype=torch.int64, device="cuda")
    step([b, a], [4, 3], tree)
    d = s.fork(b)  # forked with its drafts in place: accepting must not move rows under the fork
    rows[d] = list(rows[b])
    s.accept([b, a], [[0, 1, 3], [0, 2]])
    rows[b] = rows[b][:38] + [rows[b][38 + j] for j in (0, 1, 3)]
    rows[a] = rows[a][:38] + [rows[a][38 + j] for j in (0, 2)]
    step([a, b, d], [2, 1, 20])
    e = s.fork(d)
    rows[e] = list(rows[d])
    s.truncate(e, 33)
    rows[e] = rows[e][:33]
    step([e, d], [5, 1])
    s.free(a)
    del rows[a]
    step([b, e, d], [1, 30, 1])
    for name in (b, d, e):
        s.free(name)
    assert s.free_pages() == 60
    torch.cuda.synchronize()
    assert q.device_errors() == 0
