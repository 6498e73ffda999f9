"""GPU: reading back more rows than one per warp, so that a warp walks from row to row: over pages,
over the ends of sequences, over runs of empty and one-token ones."""
import pytest
import torch

import fp8_block_scaled_12_b200 as F
from _kv_ref import F8

pytestmark = pytest.mark.gpu


def ragged(rows, P, seed):
    """Lengths that add up to `rows`: many of none and one, some around a page, some long."""
    g = torch.Generator().manual_seed(seed)
    kinds = [0, 0, 0, 0, 1, 1, 1, 2, 7, 8, 9, P - 1, P, P + 1, 3 * P + 5, 700, 2900]
    lens, left = [], rows
    while left:
        n = min(left, kinds[int(torch.randint(0, len(kinds), (1,), generator=g))])
        lens += [n]
        left -= n
    return lens + [0, 0]


@pytest.mark.parametrize("fmt,layout", [(F.E4M3, "HND"), (F.E5M2, "NHD")])
@pytest.mark.parametrize("rows,H,D,P", [(20000, 5, 256, 8), (70001, 3, 80, 24), (70001, 8, 128, 16), (30011, 1, 16, 8),
                                        (20000, 33, 48, 32)])
def test_many_rows(cuda_device, rows, H, D, P, fmt, layout):
    """Bit for bit the rounded product of code and scale (one step of a lane holds 128 chunks of 16
    channels of k and v: 5 x 256 and 33 x 48 take two); missing pages are zeros; rows before the
    first sequence and behind the last are not written, nor is anything past `rows`."""
    pages, first, behind = 500, 5, 11
    lens = ragged(rows, P, rows + D)
    B = len(lens)
    width = -(-max(lens) // P)
    g = torch.Generator(device="cuda").manual_seed(D)
    c = F.KVCache(pages, P, H, D, fmt, layout=layout)
    c.k.copy_(torch.randint(0, 124, c.k.shape, generator=g, device="cuda").to(torch.uint8))
    c.v.copy_(torch.randint(128, 251, c.v.shape, generator=g, device="cuda").to(torch.uint8))
    c.k_scale.copy_(torch.rand(c.k_scale.shape, generator=g, device="cuda") + 0.01)
    c.v_scale.copy_(torch.rand(c.v_scale.shape, generator=g, device="cuda") * 1e-3)
    table = torch.randint(0, pages, (B, width), generator=g, device="cuda", dtype=torch.int32)
    bad = torch.rand((B, width), generator=g, device="cuda")
    table[bad < 0.05] = -1
    table[bad > 0.97] = pages
    n = torch.tensor(lens, device="cuda")
    off = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), n.cumsum(0)]) + first
    seq = torch.repeat_interleave(torch.arange(B, device="cuda"), n)
    tok = torch.arange(rows, device="cuda") + first - off[seq]
    page, row = table[seq, tok // P].long(), tok % P
    there = ((page >= 0) & (page < pages))[:, None, None]
    page = page.clamp(0, pages - 1)
    for total in (first + rows + behind, first + rows - 1234):
        ko, vo = (torch.full((total, H, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        F.fp8_kv_read(c, table, off.int(), ko, vo)
        assert F.fp8_device_error() == 0
        inside = min(rows, total - first)
        for out, codes, scales in ((ko, c.k, c.k_scale), (vo, c.v, c.v_scale)):
            x = codes[page, :, row].view(F8[fmt]).float() * scales[page, :, row][..., None]
            ref = torch.where(there, x, 0.0).to(torch.bfloat16)
            assert torch.equal(out[first:first + inside].view(torch.int16), ref[:inside].view(torch.int16))
            assert (out[:first] == 7).all() and (out[first + inside:] == 7).all()
