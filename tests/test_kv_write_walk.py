"""GPU: the writers on so many tokens that a group of lanes takes two heads and walks from token to
token: odd numbers of heads (a last group with one of its two), heads of every width, rotations of a
part, T that no step divides."""
import pytest
import torch

import fp8_block_scaled_12_b200 as F
from _kv_ref import make_cache
from test_parity_kv import EPS, check_bf16, norm_rope_ref, quant_ref, rand, tables

pytestmark = pytest.mark.gpu

# two heads a group once T x heads > 444 x 64, 32 or 16 (heads of up to 64, 128 or 256 channels)
SHAPES = [(9001, 5, 3, 64, 32), (10007, 3, 3, 16, 16), (8003, 7, 1, 80, 32), (4003, 9, 7, 128, 64),
          (2003, 5, 3, 192, 64), (1501, 3, 5, 256, 256)]


@pytest.mark.parametrize("T,Hq,Hk,D,r", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope(cuda_device, T, Hq, Hk, D, r, interleaved):
    """Against 64 bits, and bit for bit what few tokens at a time give; in place too."""
    qkv = rand((T, Hq + 2 * Hk, D), T + D)
    v = qkv[:, Hq + Hk:].clone()
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    wq, wk = rand((1, D), 5)[0], rand((1, D), 6)[0]
    pos, cs = tables(T, r, T)
    qo, ko = F.qk_norm_rope(q, k, pos, cs, wq, wk, EPS, interleaved)
    for got, x, w, what in ((qo, q, wq, "q"), (ko, k, wk, "k")):
        check_bf16(got, *norm_rope_ref(x, w, cs, pos, r, interleaved), what)
    for t in range(0, T, 300):
        part = slice(t, t + 300)
        qp, kp = F.qk_norm_rope(q[part], k[part], pos[part], cs, wq, wk, EPS, interleaved)
        assert torch.equal(qo[part], qp) and torch.equal(ko[part], kp)
    F.fp8_qk_norm_rope(q, k, pos, cs, q, k, wq, wk, EPS, interleaved)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(qkv[:, Hq + Hk:], v)
    assert F.fp8_device_error() == 0


@pytest.mark.parametrize("T,Hq,Hk,D,r", SHAPES)
def test_without_norm_or_rotation(cuda_device, T, Hq, Hk, D, r):
    q, k = rand((T, Hq, D), 1), rand((T, Hk, D), 2)
    pos, cs = tables(T, r, T)
    qo, ko = F.qk_norm_rope(q, k, pos, cs)
    check_bf16(qo, *norm_rope_ref(q, None, cs, pos, r, False), "q")
    check_bf16(ko, *norm_rope_ref(k, None, cs, pos, r, False), "k")
    qo, ko = F.qk_norm_rope(q, k, None, None)
    assert torch.equal(qo, q) and torch.equal(ko, k)


def some_slots(T, pages, P, seed):
    slots = torch.randperm(pages * P, generator=torch.Generator().manual_seed(seed)).cuda()[:T]
    slots[T // 3::7] = -1
    slots[5], slots[T - 2] = pages * P, 2 ** 40
    return slots


@pytest.mark.parametrize("layout", ["HND", "NHD", "KV"])
@pytest.mark.parametrize("fmt", [F.E4M3, F.E5M2])
@pytest.mark.parametrize("scale_fmt", [F.SCALE_FP32, F.SCALE_UE8M0])
@pytest.mark.parametrize("T,_,H,D,r", [s if s[1:4] != (7, 1, 80) else (15013, *s[1:]) for s in SHAPES])
def test_kv_write(cuda_device, layout, fmt, scale_fmt, T, _, H, D, r):
    P = 24
    pages = -(-T // P) + 2
    c = make_cache(pages, P, H, D, fmt, scale_fmt, layout)
    kv = rand((T, 2 * H, D), T, spread=2.0)
    kv[T // 2, 0] = 0
    k, v = kv[:, :H], kv[:, H:]
    slots = some_slots(T, pages, P, T)
    F.fp8_kv_write(k, v, slots, c)
    assert F.fp8_device_error() == 0
    live = ((slots >= 0) & (slots < pages * P)).cpu()
    page, row = slots.cpu()[live] // P, slots.cpu()[live] % P
    for x, codes, scales in ((k, c.k, c.k_scale), (v, c.v, c.v_scale)):
        ref_c = torch.full((pages, H, P, D), 0x7F, dtype=torch.uint8)
        ref_s = torch.full((pages, H, P), float("nan"))
        ref_c[page, :, row], ref_s[page, :, row] = quant_ref(x.cpu()[live], fmt, scale_fmt)
        assert torch.equal(codes.cpu(), ref_c)
        assert torch.equal(scales.cpu().view(torch.int32), ref_s.view(torch.int32))


@pytest.mark.parametrize("T,Hq,H,D,r", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("fmt,scale_fmt", [(F.E4M3, F.SCALE_FP32), (F.E5M2, F.SCALE_UE8M0)])
def test_fused(cuda_device, T, Hq, H, D, r, interleaved, fmt, scale_fmt):
    """Bit for bit what few tokens at a time give (one head a group), q and v what the separate calls do."""
    P = 16
    pages = -(-T // P) + 1
    qkv = rand((T, Hq + 2 * H, D), T + 1)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    wq, wk = rand((1, D), 5)[0], rand((1, D), 6)[0]
    pos, cs = tables(T, r, T)
    slots = some_slots(T, pages, P, T)
    c, few, apart = (make_cache(pages, P, H, D, fmt, scale_fmt) for _ in range(3))
    qo = F.qk_norm_rope_kv_write(q, k, v, pos, cs, slots, c, wq, wk, EPS, interleaved)
    for t in range(0, T, 300):
        part = slice(t, t + 300)
        qp = F.qk_norm_rope_kv_write(q[part], k[part], v[part], pos[part], cs, slots[part], few, wq, wk, EPS, interleaved)
        assert torch.equal(qo[part], qp)
    for a, b in ((c.k, few.k), (c.v, few.v)):
        assert torch.equal(a, b)
    for a, b in ((c.k_scale, few.k_scale), (c.v_scale, few.v_scale)):
        assert torch.equal(a.view(torch.int32), b.view(torch.int32))
    ref_q, _ = F.qk_norm_rope(q, k, pos, cs, wq, wk, EPS, interleaved)
    F.kv_write(k, v, slots, apart)
    assert torch.equal(qo, ref_q) and torch.equal(c.v, apart.v)
    assert torch.equal(c.v_scale.view(torch.int32), apart.v_scale.view(torch.int32))
    assert F.fp8_device_error() == 0


@pytest.mark.parametrize("T", [1, 37, 2003])
@pytest.mark.parametrize("interleaved", [False, True])
def test_fused_with_q_in_place(cuda_device, T, interleaved):
    """q rewritten inside the projection's output that k and v are views of: they stay."""
    Hq, H, D, r, P = 7, 3, 96, 64, 16
    qkv = rand((T, Hq + 2 * H, D), T + 9)
    before = qkv.clone()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    wq, wk = rand((1, D), 5)[0], rand((1, D), 6)[0]
    pos, cs = tables(T, r, T)
    slots = torch.arange(T, device="cuda")
    c, d = (make_cache(-(-T // P), P, H, D) for _ in range(2))
    ref = F.qk_norm_rope_kv_write(q, k, v, pos, cs, slots, c, wq, wk, EPS, interleaved)
    F.fp8_qk_norm_rope_kv_write(q, k, v, pos, cs, slots, d, q, wq, wk, EPS, interleaved)
    assert torch.equal(q, ref) and torch.equal(qkv[:, Hq:], before[:, Hq:])
    assert torch.equal(c.k, d.k) and torch.equal(c.v, d.v)
    assert F.fp8_device_error() == 0
