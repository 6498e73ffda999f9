"""GPU parity of the cache's writers and its reader: RMS norm and rotation of q and k,
quantisation into pages (bit for bit), the fused pass, and reading back."""
import pytest
import torch

import fp8_block_scaled_12_b200 as F
from _kv_ref import F8, FMAX, make_cache, make_table

pytestmark = pytest.mark.gpu
TINY = 2.0 ** -126
EPS = 1e-6


def rand(shape, seed, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda")
    return (x * torch.exp(spread * torch.randn(shape[1:], generator=g, device="cuda"))).to(torch.bfloat16)


def quant_ref(x, fmt, scale_fmt):
    """The library's FP8 rule over the last axis on the CPU: fp32 IEEE divisions, one rounding
    to the format, saturation."""
    x = x.float().cpu()
    s = (x.abs().amax(-1) / FMAX[fmt]).clamp(min=TINY)
    if scale_fmt == F.SCALE_UE8M0:
        m, e = torch.frexp(s)
        s = torch.ldexp(torch.ones_like(s), torch.where(m == 0.5, e - 1, e))
    return (x / s[..., None]).clamp(-FMAX[fmt], FMAX[fmt]).to(F8[fmt]).view(torch.uint8), s


def norm_rope_ref(x, w, cs, pos, r, interleaved, eps=EPS):
    """64-bit result and, per channel, the size of the terms it is made of."""
    n = x.double()
    if w is not None:
        n = n / torch.sqrt(n.square().mean(-1, keepdim=True) + eps) * w.double()
    y, size = n.clone(), n.abs()
    if r:
        c, s = cs[pos.clamp(0, cs.shape[0] - 1)].double()[:, None].split(r // 2, -1)
        ia = torch.arange(r // 2, device=x.device) * (2 if interleaved else 1)
        ib = ia + (1 if interleaved else r // 2)
        a, b = n[..., ia], n[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return y, size


def check_bf16(got, y, size, what):
    """One rounding to bf16 (2^-8) of an fp32 result off by at most 2^-20 of its terms, in units of
    2^-24: the sum of squares 10 (4 in a chain, 2 to join four chains, 4 over the lanes) and its
    mean and eps 2, halved by the root; the reciprocal root's 2 ulp 4; two products 2; the
    rotation 3; together 15."""
    err = (got.double() - y).abs()
    tol = 2.0 ** -8 * y.abs() + 2.0 ** -20 * size * (1 + 2.0 ** -8) + 2.0 ** -133
    assert (err <= tol).all(), f"{what}: worst {float((err / tol).max())} of the bound"


def tables(T, r, seed, max_pos=5000):
    g = torch.Generator(device="cuda").manual_seed(seed)
    pos = torch.randint(0, max_pos, (T,), generator=g, device="cuda")
    return pos, F.rope_table(max_pos, r) if r else None


SHAPES = [(1, 1, 1, 64, 64), (3, 4, 2, 128, 128), (37, 7, 1, 80, 32), (130, 2, 5, 16, 16), (65, 16, 4, 256, 256),
          (33, 8, 8, 192, 64), (9, 3, 3, 112, 112), (1000, 32, 8, 128, 128)]


@pytest.mark.parametrize("T,Hq,Hk,D,r", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_norm_rope(cuda_device, T, Hq, Hk, D, r, interleaved, norm):
    qkv = rand((T, Hq + 2 * Hk, D), T + D)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    wq, wk = (rand((1, D), 5)[0], rand((1, D), 6)[0]) if norm else (None, None)
    pos, cs = tables(T, r, T)
    qo, ko = F.qk_norm_rope(q, k, pos, cs, wq, wk, EPS, interleaved)
    for got, x, w, what in ((qo, q, wq, "q"), (ko, k, wk, "k")):
        check_bf16(got, *norm_rope_ref(x, w, cs, pos, r, interleaved), what)


def test_norm_without_rotation_and_one_weight(cuda_device):
    q, k = rand((21, 6, 96), 1), rand((21, 2, 96), 2)
    w = rand((1, 96), 3)[0]
    qo, ko = F.qk_norm_rope(q, k, None, None, wq=w)
    check_bf16(qo, *norm_rope_ref(q, w, None, None, 0, False), "q")
    assert torch.equal(ko, k)                       # neither norm nor rotation: as it was


def test_norm_rope_in_place_on_a_projection(cuda_device):
    """q and k rewritten inside the projection's output; v between them stays."""
    T, Hq, Hk, D = 77, 8, 2, 128
    qkv = rand((T, Hq + 2 * Hk, D), 4)
    before = qkv.clone()
    pos, cs = tables(T, D, 4)
    w = rand((1, D), 5)[0]
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    ref_q, ref_k = F.qk_norm_rope(q, k, pos, cs, w, w)
    F.fp8_qk_norm_rope(q, k, pos, cs, q, k, w, w)
    assert torch.equal(q, ref_q) and torch.equal(k, ref_k) and torch.equal(qkv[:, Hq + Hk:], before[:, Hq + Hk:])


def test_broadcast_inputs_and_head_major_outputs(cuda_device):
    """One token's q for all positions (a token stride of 0), outputs with heads first."""
    T, H, D = 40, 3, 64
    q = rand((1, H, D), 14).expand(T, H, D)
    k = rand((T, H, D), 15)
    pos, cs = torch.arange(T, device="cuda"), F.rope_table(64, D)
    qo = torch.empty((H, T, D), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    ko = torch.empty_like(k)
    F.fp8_qk_norm_rope(q, k, pos, cs, qo, ko)
    check_bf16(qo, *norm_rope_ref(q, None, cs, pos, D, False), "q")
    check_bf16(ko, *norm_rope_ref(k, None, cs, pos, D, False), "k")


def test_far_and_outside_positions(cuda_device):
    """Positions are taken into the table; a far one still turns by its own angle."""
    D, n = 64, 200000
    cs = F.rope_table(n, D)
    pos = torch.tensor([0, n - 1, n, -3, 131071, 2 ** 40], device="cuda")
    q, k = rand((6, 2, D), 8), rand((6, 1, D), 9)
    qo, _ = F.qk_norm_rope(q, k, pos, cs)
    check_bf16(qo, *norm_rope_ref(q, None, cs, pos, D, False), "q")
    import math
    for p in (n - 1, 131071):                       # against the angle itself, in exact integers' products
        for i in (0, 1, 31):
            a = p * 10000.0 ** (-2 * i / D)
            assert abs(float(cs[p, i]) - math.cos(a)) < 1e-7 and abs(float(cs[p, D // 2 + i]) - math.sin(a)) < 1e-7


def test_zero_and_tiny_heads(cuda_device):
    q = torch.zeros((2, 2, 128), dtype=torch.bfloat16, device="cuda")
    q[1, 1] = 2.0 ** -120
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    qo, _ = F.qk_norm_rope(q, q, None, None, w, w)
    assert torch.equal(qo[0], q[0])
    check_bf16(qo, *norm_rope_ref(q, w, None, None, 0, False), "tiny")
    qo, _ = F.qk_norm_rope(q[:1], q[:1], None, None, w, w, eps=0.0)   # 0 / 0
    assert torch.isnan(qo).all()


@pytest.mark.parametrize("layout", ["HND", "NHD", "KV"])
@pytest.mark.parametrize("fmt", [F.E4M3, F.E5M2])
@pytest.mark.parametrize("scale_fmt", [F.SCALE_FP32, F.SCALE_UE8M0])
@pytest.mark.parametrize("T,H,D,P", [(1, 1, 128, 16), (50, 3, 64, 8), (301, 8, 128, 24), (40, 2, 80, 64), (17, 5, 256, 16)])
def test_kv_write(cuda_device, layout, fmt, scale_fmt, T, H, D, P):
    pages = -(-T // P) + 2
    c = make_cache(pages, P, H, D, fmt, scale_fmt, layout)
    kv = rand((T, 2 * H, D), T, spread=2.0)
    kv[T // 2, 0] = 0                               # an empty head: the smallest scale
    k, v = kv[:, :H], kv[:, H:]
    slots = torch.randperm(pages * P, generator=torch.Generator().manual_seed(T)).cuda()[:T]
    slots[T // 3::5] = -1
    if T > 8:
        slots[3], slots[7] = pages * P, 2 ** 40     # outside the cache: skipped too
    F.fp8_kv_write(k, v, slots, c)
    torch.cuda.synchronize()
    assert F.fp8_device_error() == 0
    live = ((slots >= 0) & (slots < pages * P)).cpu()
    page, row = slots.cpu()[live] // P, slots.cpu()[live] % P
    for x, codes, scales in ((k, c.k, c.k_scale), (v, c.v, c.v_scale)):
        ref_c = torch.full((pages, H, P, D), 0x7F, dtype=torch.uint8)
        ref_s = torch.full((pages, H, P), float("nan"))
        ref_c[page, :, row], ref_s[page, :, row] = quant_ref(x.cpu()[live], fmt, scale_fmt)
        assert torch.equal(codes.cpu(), ref_c)      # untouched slots among them
        assert torch.equal(scales.cpu().view(torch.int32), ref_s.view(torch.int32))


def test_kv_write_equals_act_quant(cuda_device):
    """With D = 128 the codes and scales are act_quant's of the same rows."""
    T, H = 64, 4
    c = make_cache(T // 16, 16, H, 128)
    k, v = rand((T, H, 128), 1, 2.0), rand((T, H, 128), 2, 2.0)
    F.kv_write(k, v, torch.arange(T, device="cuda"), c)
    q, s = F.act_quant(k.reshape(T, H * 128))
    assert torch.equal(c.k.transpose(1, 2).reshape(T, H * 128), q)
    assert torch.equal(c.k_scale.transpose(1, 2).reshape(T, H), s)


@pytest.mark.parametrize("T,Hq,H,D,r", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("fmt,scale_fmt", [(F.E4M3, F.SCALE_FP32), (F.E5M2, F.SCALE_UE8M0)])
def test_fused(cuda_device, T, Hq, H, D, r, interleaved, fmt, scale_fmt):
    """q as the separate pass gives it, v as the writer does, k off its 64-bit value by one
    rounding to the format of the fp32 result."""
    P = 16
    pages = -(-T // P) + 1
    qkv = rand((T, Hq + 2 * H, D), T + 1)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    wq, wk = rand((1, D), 5)[0], rand((1, D), 6)[0]
    pos, cs = tables(T, r, T)
    slots = torch.randperm(pages * P, generator=torch.Generator().manual_seed(T)).cuda()[:T]
    if T > 2:
        slots[1] = -1
    c, c2 = (make_cache(pages, P, H, D, fmt, scale_fmt) for _ in range(2))
    qo = F.qk_norm_rope_kv_write(q, k, v, pos, cs, slots, c, wq, wk, EPS, interleaved)
    ref_q, _ = F.qk_norm_rope(q, k, pos, cs, wq, wk, EPS, interleaved)
    F.kv_write(k, v, slots, c2)
    assert F.fp8_device_error() == 0
    assert torch.equal(qo, ref_q)
    assert torch.equal(c.v, c2.v) and torch.equal(c.v_scale.view(torch.int32), c2.v_scale.view(torch.int32))
    live = slots >= 0
    page, row = slots[live] // P, slots[live] % P
    y, size = norm_rope_ref(k, wk, cs, pos, r, interleaved)
    y, size = y[live], size[live]
    s = c.k_scale[page, :, row].double()
    exact_s = y.abs().amax(-1) / FMAX[fmt]
    fp32 = 2.0 ** -20 * size.amax(-1) / FMAX[fmt]   # what the fp32 result's amax may be off by
    if scale_fmt == F.SCALE_FP32:
        assert ((s - exact_s).abs() <= fp32 + 2.0 ** -23 * exact_s).all()
    else:                                           # the power of two at or above, but for a near tie
        m, _ = torch.frexp(s)
        assert (m == 0.5).all()
        assert ((s >= exact_s - fp32) & (s / 2 < exact_s + fp32)).all()
    x = y / s[..., None]
    err = (c.k[page, :, row].view(F8[fmt]).double() - x).abs()
    half, least = (2.0 ** -4, 2.0 ** -10) if fmt == F.E4M3 else (2.0 ** -3, 2.0 ** -17)
    tol = torch.maximum(half * x.abs(), torch.full_like(x, least)) * (1 + 2.0 ** -10) + \
        2.0 ** -19 * size / s[..., None]
    assert (err <= tol).all(), float((err / tol).max())
    untouched = torch.ones((pages, P), dtype=torch.bool, device="cuda")
    untouched[page, row] = False
    assert (c.k.transpose(1, 2)[untouched] == 0x7F).all()


@pytest.mark.parametrize("layout", ["HND", "NHD", "KV"])
@pytest.mark.parametrize("fmt", [F.E4M3, F.E5M2])
@pytest.mark.parametrize("H,D,P", [(1, 128, 16), (8, 128, 64), (3, 80, 24), (5, 256, 8), (2, 16, 128)])
def test_kv_read(cuda_device, layout, fmt, H, D, P):
    """bf16 of the fp32 product of code and scale, rounded once; nothing outside the ranges."""
    lens = [5, 0, 130, 1, 64, 301]
    pages = sum(-(-n // P) for n in lens) + 1
    c = make_cache(pages, P, H, D, fmt, layout=layout)
    table = make_table(lens, P, pages, D)
    g = torch.Generator(device="cuda").manual_seed(D)
    c.k.copy_(torch.randint(0, 124, c.k.shape, generator=g, device="cuda").to(torch.uint8))
    c.v.copy_(torch.randint(128, 251, c.v.shape, generator=g, device="cuda").to(torch.uint8))
    c.k_scale.copy_(torch.rand(c.k_scale.shape, generator=g, device="cuda") + 0.01)
    c.v_scale.copy_(torch.rand(c.v_scale.shape, generator=g, device="cuda") * 1e-3)
    first = 3                                       # rows before the first and behind the last range
    off = torch.tensor([0] + lens).cumsum(0).add(first).int().cuda()
    rows = int(off[-1]) + 4
    ko = torch.full((rows, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    table[5, 0] = -1                                # a page that is not there
    F.fp8_kv_read(c, table, off, ko, vo)
    torch.cuda.synchronize()
    for out, codes, scales in ((ko, c.k, c.k_scale), (vo, c.v, c.v_scale)):
        ref = torch.full_like(out, 7.0)
        for b, n in enumerate(lens):
            tok = torch.arange(n, device="cuda")
            pg, rw = table[b].long()[tok // P], tok % P
            there = (pg >= 0)[:, None, None]
            pg = pg.clamp(min=0)
            x = codes[pg, :, rw].view(F8[fmt]).float() * scales[pg, :, rw][..., None]
            ref[int(off[b]):int(off[b + 1])] = torch.where(there, x, 0.0).to(torch.bfloat16)
        assert torch.equal(out, ref)


def test_kv_read_beyond_the_table(cuda_device):
    c = make_cache(4, 8, 1, 16)
    c.k.fill_(0x38)
    c.k_scale.fill_(1.0)
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 12], dtype=torch.int32, device="cuda")
    ko, _ = F.kv_read(c, table, off, 12)
    assert (ko[:8] == 1).all() and (ko[8:] == 0).all()


def test_kv_read_of_offsets_far_below_zero(cuda_device):
    """The host cannot check device offsets: token numbers past 32 bits count as beyond the table."""
    c = make_cache(4, 16, 2, 64)
    table = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    off = torch.tensor([-2 ** 31, 12], dtype=torch.int32, device="cuda")
    ko, vo = F.kv_read(c, table, off, 12)
    assert F.fp8_device_error() == 0
    assert (ko == 0).all() and (vo == 0).all()
