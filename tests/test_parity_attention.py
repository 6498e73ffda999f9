"""GPU parity of the paged decode attention against a plain 64-bit form: head layouts, page
sizes, lengths from none to long ones, windows, pages that are not there, and whatever
bytes lie beyond the tokens that count (the caches here are NaN wherever nothing was written)."""
import math

import pytest
import torch

import fp8_block_scaled_12_b200 as F
from _kv_ref import attention_ref, check_attention, fill_cache, make_cache, make_table

pytestmark = pytest.mark.gpu


def case(lens, H, G, D, P, fmt=F.E4M3, layout="HND", window=0, seed=0, k_gain=1.0, scale=None):
    dev = "cuda"
    pages = sum(-(-n // P) for n in lens) + 2
    c = make_cache(pages, P, H, D, fmt, layout=layout)
    table = make_table(lens, P, pages, seed)
    kv = fill_cache(c, table, lens, seed, k_gain)
    g = torch.Generator(device=dev).manual_seed(seed + 1)
    q = torch.randn((len(lens), H * G, D), generator=g, device=dev).to(torch.bfloat16)
    n = torch.tensor(lens, dtype=torch.int32, device=dev)
    out, lse = F.paged_attention(q, c, table, n, scale=scale, window=window, return_lse=True)
    assert F.fp8_device_error() == 0
    ref, rlse, tol, ltol = attention_ref(q, kv, scale, window)
    check_attention(out, ref, tol, "out")
    empty = torch.isinf(rlse)
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty)
    check_attention(lse[~empty], rlse[~empty], ltol[~empty], "lse")
    assert (out[empty] == 0).all()
    return c, table, q, n, out


def test_one_tile(cuda_device):
    case([128], 1, 8, 128, 128)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 127, 129, 255, 256, 257, 1000])
def test_lengths(cuda_device, n):
    case([n], 2, 4, 128, 16, seed=n)


def test_ragged_batch_with_empty_rows(cuda_device):
    case([0, 1, 700, 0, 128, 3, 2049, 64, 0], 2, 4, 128, 16)


def test_only_empty_rows(cuda_device):
    case([0, 0, 0], 2, 4, 64, 16)


@pytest.mark.parametrize("G", [1, 2, 3, 7, 8, 9, 12, 16, 17, 24, 40])
def test_head_groups(cuda_device, G):
    case([300, 5], 2, G, 128, 32, seed=G)


@pytest.mark.parametrize("D", [16, 48, 64, 80, 112, 128, 144, 192, 256])
@pytest.mark.parametrize("G", [4, 16])
def test_head_dims(cuda_device, D, G):
    case([513, 100], 3, G, D, 16, seed=D)


@pytest.mark.parametrize("P", [8, 16, 24, 32, 48, 64, 120, 128, 136, 256, 1024])
def test_page_sizes(cuda_device, P):
    case([1025, 77, P, P + 1], 2, 4, 64, P, seed=P)


@pytest.mark.parametrize("layout", ["HND", "NHD", "KV"])
@pytest.mark.parametrize("fmt", [F.E4M3, F.E5M2])
@pytest.mark.parametrize("D", [96, 256])
def test_layouts_and_formats(cuda_device, layout, fmt, D):
    case([333, 128, 9], 3, 5, D, 16, fmt, layout)


@pytest.mark.parametrize("window", [1, 5, 127, 128, 129, 500, 100000])
def test_windows(cuda_device, window):
    case([1000, 3, 128, 0, 400], 2, 4, 128, 16, window=window)


def test_many_rows_more_than_the_gpu_holds(cuda_device):
    case([(37 * i) % 401 for i in range(150)], 4, 2, 64, 16)


def test_one_long_row_is_split_over_the_gpu(cuda_device):
    case([40000], 1, 8, 128, 64, seed=3)


def test_rows_cut_by_the_ranges(cuda_device):
    """Lengths that put the ranges' borders inside rows and leave some CTAs several rows."""
    case([5000, 1, 3000 - 1, 130, 12000, 0, 260, 7777], 4, 8, 128, 16, seed=5)


@pytest.mark.parametrize("H,G,D,P", [(8, 4, 128, 16), (4, 12, 64, 32), (4, 4, 256, 64)])
def test_many_tiles_a_worker(cuda_device, H, G, D, P):
    """Ragged rows over the whole GPU, several tiles and several rows a worker, the two
    warpgroups of a CTA with unequal shares."""
    lens = [max(1, 6000 - int(6000 * ((0.6180339887498949 * i) % 1.0))) for i in range(40)]
    c, table, q, n, out = case(lens, H, G, D, P, seed=11)
    for _ in range(3):
        assert torch.equal(F.paged_attention(q, c, table, n), out)


@pytest.mark.parametrize("gain", [1e-3, 30.0, 300.0])
def test_flat_and_peaked_softmax(cuda_device, gain):
    """Scores from almost equal to hundreds of nats apart."""
    case([2000, 129], 2, 8, 128, 16, k_gain=gain, seed=7)


def test_negative_and_zero_scale(cuda_device):
    case([300], 2, 4, 64, 16, scale=-0.3)
    case([300], 2, 4, 64, 16, scale=0.0)


def test_value_scales_over_many_decades(cuda_device):
    """One token with nearly all of the probability and a tiny value, the rest the other way
    round: the sum keeps both."""
    lens, H, G, D, P = [1500], 1, 8, 128, 16
    c = make_cache(100, P, H, D)
    table = make_table(lens, P, 100, 0)
    fill_cache(c, table, lens, 0)
    first = table[0, 0].item()
    c.k_scale[first, :, 0] *= 40
    c.v_scale[first, :, 0] = 2.0 ** -126
    c.v_scale[table[0, 7].item(), :, 3] *= 1e20
    c.v_scale[table[0, 50].item()] *= 1e-15
    kv = []
    tok = torch.arange(lens[0], device="cuda")
    pg, rw = table[0].long()[tok // P], tok % P
    for x, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
        kv.append(x[pg, :, rw].view(torch.float8_e4m3fn).double() * s[pg, :, rw].double()[..., None])
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn((1, G, D), generator=g, device="cuda").to(torch.bfloat16)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = F.paged_attention(q, c, table, n)
    ref, _, tol, _ = attention_ref(q, [tuple(kv)])
    check_attention(out, ref, tol, "out")


def test_pages_outside_the_cache_are_left_out(cuda_device):
    lens, P = [1000, 40, 16], 16
    c = make_cache(80, P, 2, 128)
    table = make_table(lens, P, 80, 1)
    kv = fill_cache(c, table, lens, 1)
    skip = [torch.zeros(n, dtype=torch.bool, device="cuda") for n in lens]
    for b, p, bad in ((0, 0, -1), (0, 7, 80), (0, 8, 2 ** 31 - 1), (0, 62, -2 ** 31), (1, 1, -1), (2, 0, 99999)):
        table[b, p] = bad
        skip[b][p * P:(p + 1) * P] = True
    q = torch.randn((3, 8, 128), device="cuda").to(torch.bfloat16)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = F.paged_attention(q, c, table, n, return_lse=True)
    ref, rlse, tol, ltol = attention_ref(q, kv, skip=skip)
    check_attention(out, ref, tol, "out")
    check_attention(lse[:2], rlse[:2], ltol[:2], "lse")
    assert (out[2] == 0).all() and (lse[2] == -math.inf).all()


def test_lengths_outside_the_table(cuda_device):
    """A length beyond the table counts as the table's, a negative one as none."""
    P = 16
    c = make_cache(20, P, 2, 64)
    table = make_table([128, 128], P, 20, 2)
    kv = fill_cache(c, table, [128, 128], 2)
    q = torch.randn((2, 4, 64), device="cuda").to(torch.bfloat16)
    out = F.paged_attention(q, c, table, torch.tensor([2 ** 31 - 1, -5], dtype=torch.int32, device="cuda"))
    ref, _, tol, _ = attention_ref(q, [kv[0], (kv[1][0][:0], kv[1][1][:0])])
    check_attention(out, ref, tol, "out")
    none = F.paged_attention(q, c, table[:, :0], torch.tensor([5, 0], dtype=torch.int32, device="cuda"))
    assert (none == 0).all()


def test_strided_queries_and_table(cuda_device):
    """q as a view of a wider projection, rows of a wider table."""
    lens, P, H, G, D = [300, 20, 129], 16, 2, 4, 128
    c = make_cache(60, P, H, D)
    table = make_table(lens, P, 60, 4, width=70)
    kv = fill_cache(c, table, lens, 4)
    qkv = torch.randn((3, H * G + 2 * H, D), device="cuda").to(torch.bfloat16)
    q = qkv[:, :H * G]
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = F.paged_attention(q, c, table[:, :30], n)
    ref, _, tol, _ = attention_ref(q.contiguous(), kv)
    check_attention(out, ref, tol, "out")
    heads_first = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(F.paged_attention(heads_first, c, table, n), out)


def test_non_finite_values_that_count(cuda_device):
    """A NaN or infinite query makes its head NaN and no other; a NaN code of v its channel."""
    lens, P, H, G, D = [200], 16, 2, 4, 64
    c = make_cache(20, P, H, D)
    table = make_table(lens, P, 20, 6)
    fill_cache(c, table, lens, 6)
    q = torch.randn((1, H * G, D), device="cuda").to(torch.bfloat16)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    clean = F.paged_attention(q, c, table, n)
    q2 = q.clone()
    q2[0, 1, 5] = math.nan
    q2[0, 6, 0] = math.inf
    out = F.paged_attention(q2, c, table, n)
    for h in range(H * G):
        if h in (1, 6):
            assert torch.isnan(out[0, h]).all()
        else:
            assert torch.equal(out[0, h], clean[0, h])
    c.v[table[0, 3].item(), 1, 2, 17] = 0x7F
    out = F.paged_attention(q, c, table, n)
    assert torch.isnan(out[0, G:, 17]).all()
    out[0, G:, 17] = clean[0, G:, 17]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_non_finite_value_scales_that_count(cuda_device, bad):
    """A token whose v scale is not finite makes the heads that read it NaN in every channel,
    also those where its code is zero, and no other head."""
    lens, P, H, G, D = [300], 16, 2, 4, 64
    c = make_cache(20, P, H, D)
    table = make_table(lens, P, 20, 7)
    fill_cache(c, table, lens, 7)
    q = torch.randn((1, H * G, D), device="cuda").to(torch.bfloat16)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    clean = F.paged_attention(q, c, table, n)
    page = table[0, 9].item()
    c.v[page, 1, 3, :8] = 0
    c.v_scale[page, 1, 3] = bad
    out = F.paged_attention(q, c, table, n)
    assert F.fp8_device_error() == 0
    assert torch.isnan(out[0, G:]).all()
    assert torch.equal(out[0, :G], clean[0, :G])


@pytest.mark.parametrize("H,G,D,P", [(8, 4, 128, 16), (2, 8, 128, 8), (2, 16, 64, 16), (4, 2, 192, 32)])
def test_many_random_batches(cuda_device, H, G, D, P):
    """Fifty batches of random lengths (partly masked tiles at the beginning, the middle and the end
    of the workers' ranges): every wait ends, and a second call gives the same bits."""
    g = torch.Generator().manual_seed(H * G + D)
    pages = 8000
    c = make_cache(pages, P, H, D)
    for t in (c.k, c.v):
        t.copy_(torch.randint(0, 124, t.shape, device="cuda").to(torch.uint8))
    c.k_scale.uniform_(1e-4, 2e-3)
    c.v_scale.uniform_(1e-3, 1e-2)
    for i in range(50):
        B = int(torch.randint(1, 70, (1,), generator=g))
        lens = (torch.rand(B, generator=g) ** 3 * (pages * P // max(B, 16))).int()
        width = max(1, int(-(-lens.max() // P)))
        table = torch.randint(0, pages, (B, width), generator=g, dtype=torch.int32).cuda()
        q = torch.randn((B, H * G, D), device="cuda").to(torch.bfloat16)
        n = lens.cuda()
        window = int(torch.randint(0, 3, (1,), generator=g)) * 333
        out = F.paged_attention(q, c, table, n, window=window)
        again = F.paged_attention(q, c, table, n, window=window)
        assert F.fp8_device_error() == 0, (i, lens.tolist())
        assert torch.isfinite(out).all() and torch.equal(out, again), (i, lens.tolist())


def test_same_call_same_bits(cuda_device):
    c, table, q, n, out = case([5000, 1, 2999, 130, 900], 4, 8, 128, 16, seed=8)
    for _ in range(5):
        assert torch.equal(F.paged_attention(q, c, table, n), out)


@pytest.mark.parametrize("B,H,L", [(80, 8, 700), (300, 2, 1), (600, 1, 300), (37, 8, 2000)])
def test_rows_around_the_number_of_workers_any_workspace(cuda_device, B, H, L):
    """More rows than workers and fewer, cut and whole: what the workspace holds before does not
    matter, not even what looks like an entry of an earlier call."""
    G, D, P = 4, 64, 16
    lens = [(i * 7919) % (L + 1) for i in range(B)]
    c, table, q, n, out = case(lens, H, G, D, P, seed=9)
    ws = torch.empty(F.paged_attention_ws_bytes(B, H * G, c), dtype=torch.uint8, device="cuda")
    for fill in (0, 1, 0x7F, 0xFF):
        ws.fill_(fill)
        again = torch.full_like(out, math.nan)
        F.fp8_paged_attention(q, c, table, n, again, ws)
        assert torch.equal(again, out)
        F.fp8_paged_attention(q, c, table, torch.flip(n, [0]).contiguous(), again, ws)     # other cuts, then the same
        F.fp8_paged_attention(q, c, table, n, again, ws)
        assert torch.equal(again, out)
    assert F.fp8_device_error() == 0
