"""GPU: attention over value scales that lie decades apart.  What a token adds to the output is its
probability times its value scale times its codes, so a large scale with hardly any probability must
not cost the others their bits, nor a small one with nearly all of it its own."""
import math

import pytest
import torch

import fp8_block_scaled_12_b200 as F
from _kv_ref import F8, make_cache, make_table

pytestmark = pytest.mark.gpu
TILE = 128


def reference(q, c, table, lens):
    """(out, bound, lse, bound) in 64 bits, with a bound made of what each token contributes.

    A score is off by ds (D + 8 roundings of 2^-24 of its absolute sum, and q by 2^-21 of its largest
    element), so its probability by ds relative, by 2^-22 for the exponential and for each running
    factor, and by 2^-17 for exponents of up to 128 binades (2^-24 of a difference of two of them).
    The weights p sv are held to 2^-17 relative, or to 2^-29 of the largest of their tile.  An error
    d_t of p_t moves out by p_t d_t (|v_t| + |out|).  bf16 rounds by 2^-8 (at least half of 2^-133)."""
    B, Hq, D = q.shape
    H, G = c.heads, Hq // c.heads
    out = torch.zeros((B, Hq, D), dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=q.device)
    ltol = torch.zeros_like(lse)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        tok = torch.arange(n, device=q.device)
        pg, rw = table[b].long()[tok // c.page_size], tok % c.page_size
        k = c.k[pg, :, rw].view(F8[c.fmt]).double() * c.k_scale[pg, :, rw].double()[..., None]     # [n, H, D]
        code, sv = c.v[pg, :, rw].view(F8[c.fmt]).double(), c.v_scale[pg, :, rw].double()
        x = q[b].double().view(H, G, D)
        s = torch.einsum("hgd,lhd->hgl", x, k) / math.sqrt(D)
        sabs = torch.einsum("hgd,lhd->hgl", x.abs(), k.abs()) / math.sqrt(D)
        p = torch.softmax(s, -1)
        w = p * sv.T[:, None]
        o = torch.einsum("hgl,lhd->hgd", w, code)
        ds = (D + 8) * 2.0 ** -24 * sabs + 2.0 ** -21 * x.abs().amax(-1)[..., None] * k.abs().sum(-1).T[:, None] / math.sqrt(D)
        tiles = -(-n // TILE)
        dp = ds + 2.0 ** -22 * (1 + tiles) + 2 * 2.0 ** -17
        t = torch.einsum("hgl,lhd->hgd", w * dp, code.abs()) + (p * dp).sum(-1)[..., None] * o.abs()
        for i in range(tiles):
            part = slice(i * TILE, (i + 1) * TILE)
            t += 2.0 ** -29 * w[..., part].amax(-1)[..., None] * code[part].abs().sum(0)[:, None]
        out[b], tol[b] = o.reshape(Hq, D), (t * (1 + 2.0 ** -8) + 2.0 ** -8 * o.abs() + 2.0 ** -134).reshape(Hq, D)
        lse[b] = torch.logsumexp(s, -1).reshape(Hq)
        ltol[b] = ((p * dp).sum(-1) + 2.0 ** -22).reshape(Hq) + 2.0 ** -22 * lse[b].abs()
    return out, tol, lse, ltol


def check(q, c, table, lens):
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = F.paged_attention(q, c, table, n, return_lse=True)
    assert F.fp8_device_error() == 0
    ref, tol, rlse, ltol = reference(q, c, table, lens)
    assert torch.isfinite(out).all()
    err = (out.double() - ref).abs()
    some = torch.tensor(lens, device="cuda") > 0
    # the bound is worth something: an output of zeros is outside it for most channels of every head
    assert ((ref.abs() > tol)[some].double().mean(-1) > 0.8).all()
    assert (err <= tol).all(), f"{int((err > tol).sum())} of {err.numel()} beyond the bound, worst " \
        f"{float((err / tol)[some].max())} times"
    assert ((lse.double() - rlse).abs() <= ltol)[some].all()


def normal(lens, H, G, D, P, fmt, seed):
    """Ordinary contents: values of size 1, scores of size 1/2."""
    pages = sum(-(-n // P) for n in lens) + 1
    c = make_cache(pages, P, H, D, fmt)
    table = make_table(lens, P, pages, seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for b, n in enumerate(lens):
        tok = torch.arange(n, device="cuda")
        pg, rw = table[b].long()[tok // P], tok % P
        for codes, scales in ((c.k, c.k_scale), (c.v, c.v_scale)):
            x = torch.randn((n, H, D), generator=g, device="cuda") * 16
            codes[pg, :, rw] = x.clamp(-448, 448).to(F8[fmt]).view(torch.uint8)
            scales[pg, :, rw] = torch.exp(0.5 * torch.randn((n, H), generator=g, device="cuda")) / 32
    return c, table, g


def one_apart(c, table, g, G, token, nats, v_factor, b=0):
    """Queries along +-1 vectors, and the k of `token` along them so that its score lies about `nats`
    above the others' (below for a negative number) for all heads; its v scale times v_factor."""
    H, D, P = c.heads, c.head_dim, c.page_size
    u = torch.randint(0, 2, (H, D), generator=g, device="cuda") * 2.0 - 1
    q = (u[:, None] + 0.25 * torch.randn((H, G, D), generator=g, device="cuda")).reshape(1, H * G, D)
    page, row = int(table[b, token // P]), token % P
    c.k[page, :, row] = (u * math.copysign(8, nats)).to(F8[c.fmt]).view(torch.uint8)
    c.k_scale[page, :, row] = abs(nats) * math.sqrt(D) / (8 * D)
    c.v_scale[page, :, row] *= v_factor
    return q.to(torch.bfloat16)


SHAPES = [(1, 8, 128, 16, F.E4M3), (2, 3, 64, 32, F.E5M2), (2, 12, 128, 16, F.E4M3), (1, 5, 192, 8, F.E4M3)]


@pytest.mark.parametrize("H,G,D,P,fmt", SHAPES)
@pytest.mark.parametrize("factor", [1e7, 1e10, 1e20])
@pytest.mark.parametrize("n", [100, 1500])
def test_a_large_scale_without_probability(cuda_device, H, G, D, P, fmt, factor, n):
    c, table, g = normal([n], H, G, D, P, fmt, 1)
    q = one_apart(c, table, g, G, 37, -100.0, factor)
    check(q, c, table, [n])


@pytest.mark.parametrize("H,G,D,P,fmt", SHAPES)
@pytest.mark.parametrize("nats,factor", [(20.0, 1e-6), (40.0, 1e-12), (60.0, 1e-20)])
@pytest.mark.parametrize("n", [100, 1500])
def test_a_small_scale_with_nearly_all_probability(cuda_device, H, G, D, P, fmt, nats, factor, n):
    c, table, g = normal([n], H, G, D, P, fmt, 2)
    q = one_apart(c, table, g, G, 37, nats, factor)
    check(q, c, table, [n])


@pytest.mark.parametrize("H,G,D,P,fmt", SHAPES)
@pytest.mark.parametrize("binades", [20, 44])
def test_scales_spread_over_a_tile(cuda_device, H, G, D, P, fmt, binades):
    """Every token with a scale of its own, up to 2 x binades apart, rows of one worker and cut ones."""
    lens = [700, 1, 3, 128, 0, 300, 2500]
    c, table, g = normal(lens, H, G, D, P, fmt, 3)
    e = torch.rand(c.v_scale.shape, generator=g, device="cuda") * (2 * binades) - binades
    c.v_scale.mul_(torch.exp2(e))
    q = torch.randn((len(lens), H * G, D), generator=g, device="cuda") * 8
    check(q.to(torch.bfloat16), c, table, lens)


@pytest.mark.parametrize("H,G,D,P,fmt", SHAPES)
@pytest.mark.parametrize("binades", [5, 38])
def test_scales_that_differ_between_tiles(cuda_device, H, G, D, P, fmt, binades):
    """The tiles' references lie apart by their scales as well as by their scores: a tile of small
    scales still has its share of the probability, in one worker's sums and in the join's."""
    lens = [128 * 40 + 17, 384, 128 * 9]
    c, table, g = normal(lens, H, G, D, P, fmt, 6)
    for b, n in enumerate(lens):
        tok = torch.arange(n, device="cuda")
        e = ((tok // TILE) * 7 % 3 - 1) * binades
        c.v_scale[table[b].long()[tok // P], :, tok % P] *= torch.exp2(e.float())[:, None]
    q = torch.randn((len(lens), H * G, D), generator=g, device="cuda").to(torch.bfloat16)
    check(q, c, table, lens)


@pytest.mark.parametrize("scale", [2.0 ** -126, 3.0 * 2.0 ** -120, 2.0 ** -100, 2.0 ** 90, 2.0 ** 118])
def test_all_scales_small_or_large(cuda_device, scale):
    """The smallest scale that the writers store, and values near both ends of bf16."""
    lens = [700, 5]
    c, table, g = normal(lens, 2, 4, 128, 16, F.E4M3, 4)
    c.v_scale.copy_(torch.where(torch.isnan(c.v_scale), c.v_scale, scale))
    q = torch.randn((2, 8, 128), generator=g, device="cuda").to(torch.bfloat16)
    check(q, c, table, lens)


@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_a_value_scale_that_is_not_finite_leaves_the_statistics(cuda_device, bad):
    """It makes its row NaN, but lse is a matter of the scores alone."""
    c, table, g = normal([300], 2, 4, 64, 16, F.E4M3, 5)
    q = torch.randn((1, 8, 64), generator=g, device="cuda").to(torch.bfloat16)
    n = torch.tensor([300], dtype=torch.int32, device="cuda")
    page = int(table[0, 9])
    c.v_scale[page, 1, 3] = bad
    out, lse = F.paged_attention(q, c, table, n, return_lse=True)
    assert F.fp8_device_error() == 0
    assert torch.isnan(out[0, 4:]).all() and torch.isfinite(out[0, :4]).all()
    c.v_scale[page, 1, 3] = 1.0
    _, _, rlse, ltol = reference(q, c, table, [300])
    assert ((lse.double() - rlse).abs() <= ltol).all()
