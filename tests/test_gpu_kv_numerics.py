"""The K/V cache operators over values far from one: tiny groups, groups of different scale, one position that
outweighs a hundred thousand others."""
import math

import pytest
import torch

import bit_quantized_gemm_qmm_b200 as q
import kv_reference as ref
from test_gpu_kv import BF, HF, gen, ints

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
