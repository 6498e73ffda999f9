"""Plain 64-bit restatements of the paged-cache operators (test-side only), and the error
bounds that their arithmetic allows."""
import math

import torch

import fp8_block_scaled_12_b200 as F

FMAX = {F.E4M3: 448.0, F.E5M2: 57344.0}
F8 = {F.E4M3: torch.float8_e4m3fn, F.E5M2: torch.float8_e5m2}
NAN_CODE = {F.E4M3: 0x7F, F.E5M2: 0x7F}


def make_cache(pages, P, H, D, fmt=F.E4M3, scale_fmt=F.SCALE_FP32, layout="HND", device="cuda"):
    """A cache whose every byte is a NaN code and every scale a NaN: whatever a reader uses
    without being allowed to shows up."""
    if layout == "KV":                        # k and v of a page side by side in one allocation
        both = torch.empty((pages, 2, P, H, D), dtype=torch.uint8, device=device).permute(1, 0, 3, 2, 4)
        sc = [torch.empty((pages, H, P), dtype=torch.float32, device=device) for _ in range(2)]
        c = F.KVCache.wrap(both[0], both[1], sc[0], sc[1], fmt, scale_fmt)
    else:
        c = F.KVCache(pages, P, H, D, fmt, scale_fmt, layout, device)
    c.k.fill_(NAN_CODE[fmt])
    c.v.fill_(NAN_CODE[fmt])
    c.k_scale.fill_(math.nan)
    c.v_scale.fill_(math.nan)
    return c


def fill_cache(c, table, lens, seed, k_gain=1.0):
    """Valid contents for tokens [0, lens[b]) of every sequence; everything else stays NaN.
    Returns 64-bit k, v per sequence: [len, H, D]."""
    g = torch.Generator(device=c.device).manual_seed(seed)
    out = []
    for b, n in enumerate(lens):
        tok = torch.arange(n, device=c.device)
        page, row = table[b].long()[tok // c.page_size], tok % c.page_size
        kv = []
        for codes, scales, gain in ((c.k, c.k_scale, k_gain), (c.v, c.v_scale, 1.0)):
            x = torch.randn((n, c.heads, c.head_dim), generator=g, device=c.device) * (FMAX[c.fmt] / 4)
            q = x.clamp(-FMAX[c.fmt], FMAX[c.fmt]).to(F8[c.fmt])
            s = torch.exp(torch.randn((n, c.heads), generator=g, device=c.device)) * (4 * gain / FMAX[c.fmt])
            codes[page, :, row] = q.view(torch.uint8)
            scales[page, :, row] = s
            kv.append(q.double() * s.double()[..., None])
        out.append(tuple(kv))
    return out


def make_table(lens, P, pages, seed, device="cuda", width=None):
    """Page ids of every sequence, drawn without repetition; entries past a sequence's last
    page are out of range on purpose."""
    need = [-(-n // P) for n in lens]
    width = width or max(1, max(need, default=1))
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).int()
    assert sum(need) <= pages
    t = torch.full((len(lens), width), 2 ** 31 - 1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = perm[at:at + n]
        at += n
    return t.to(device)


def attention_ref(q, kv, scale=None, window=0, skip=None):
    """(out, lse, bound of out, bound of lse) in 64 bits for bf16 q [B, Hq, D] and per-sequence
    (k, v) [len, H, D].  `skip[b]`: tokens left out.

    The bound: a score is a sum of D exact products of E4M3 pieces with fp32 accumulation (D + 8
    roundings of 2^-24 of the absolute sum), of q off by at most 2^-21 of its largest element;
    a probability adds 2^-22 (exponential) and 2^-17 (its pieces), each of the n tiles' running
    factors 2^-22; weights are held to 2^-30 of the tile's largest, 128 of them: 2^-23 of the
    largest |v|.  Relative errors of the probabilities enter numerator and denominator.  The
    output is rounded to bf16: 2^-8 relative."""
    B, Hq, D = q.shape
    scale = 1 / math.sqrt(D) if scale is None else scale
    out = torch.zeros((B, Hq, D), dtype=torch.float64, device=q.device)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=q.device)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    for b, (k, v) in enumerate(kv):
        n = k.shape[0]
        keep = torch.ones(n, dtype=torch.bool, device=q.device)
        if window:
            keep[:max(0, n - window)] = False
        if skip is not None:
            keep &= ~skip[b]
        k, v = k[keep], v[keep]
        if k.shape[0] == 0:
            continue
        H = k.shape[1]
        x = q[b].double().view(H, -1, D)
        s = torch.einsum("hgd,lhd->hgl", x, k) * scale
        p = torch.softmax(s, -1)
        out[b] = torch.einsum("hgl,lhd->hgd", p, v).reshape(Hq, D)
        lse[b] = torch.logsumexp(s, -1).reshape(Hq)
        sabs = torch.einsum("hgd,lhd->hgl", x.abs(), k.abs()) * abs(scale)
        qmax = x.abs().amax(-1)[..., None]
        ds = (D + 8) * 2.0 ** -24 * sabs + 2.0 ** -21 * qmax * k.abs().sum(-1).T[:, None] * abs(scale)
        tiles = n // 128 + 2
        dp = ds.amax(-1) + 2.0 ** -22 * (1 + tiles) + 2.0 ** -17
        mass = torch.einsum("hgl,lhd->hgd", p, v.abs())
        t = 2 * dp[..., None] * mass + 2.0 ** -23 * v.abs().amax()
        tol[b] = t.reshape(Hq, D) * (1 + 2.0 ** -8) + 2.0 ** -8 * out[b].abs()
        ltol[b] = (ds.amax(-1) + 2.0 ** -22 * (1 + tiles) + (tiles + 16) * 2.0 ** -24).reshape(Hq) + \
            2.0 ** -22 * (1 + lse[b].abs())
    return out, lse, tol, ltol


def check_attention(got, ref, tol, what):
    if got.numel() == 0:
        return
    assert torch.isfinite(got).all(), f"{what}: not finite at {(~torch.isfinite(got)).nonzero()[:4].tolist()}"
    err = (got.double() - ref).abs()
    bad = err > tol
    i = int((err / tol.clamp(min=1e-300)).argmax())
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst " \
        f"{float(got.flatten()[i])} against {float(ref.flatten()[i])} +- {float(tol.flatten()[i])}, first at " \
        f"{bad.nonzero()[:4].tolist()}"
