"""The quantised paged key-value cache and what reads and writes it: cases for measurement.

Five operators of a decoder layer around an FP8 cache of pages (codes [pages, heads, page, dim] and one
fp32 scale per token and head):

  qk_norm_rope           RMS norm of every head of q and k, and the position rotation
  kv_write               k and v quantised into the slots of their tokens
  qk_norm_rope_kv_write  both in one pass: q comes back in bf16, k and v go to the cache
  kv_read                the pages of a batch of sequences back as bf16 rows
  paged_attention        one new token per sequence against its pages

`run` computes them in elementary torch operations (own = False) or calls the library (own = True).
"""
import math

import torch

own = False

EPS = 1e-6
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TINY = 2.0 ** -126
POSITIONS = 8192          # rows of the rotation's table


# ------------------------------------------------------------------ cases
def _write(op, name, t, hq, hkv, d, r, page, fmt="e4m3", scale="fp32", layout="HND", interleaved=False):
    return dict(name=name, op=op, t=t, hq=hq, hkv=hkv, d=d, r=r, page=page, fmt=fmt, scale=scale, layout=layout,
                interleaved=interleaved)


def _read(op, name, b, longest, hq, hkv, d, page, fmt="e4m3", layout="HND", window=0):
    return dict(name=name, op=op, b=b, longest=longest, hq=hq, hkv=hkv, d=d, page=page, fmt=fmt, layout=layout,
                window=window)


def listed():
    return [
        # a prompt of 4096 tokens before its own (bf16) attention: q and k in place of the projection's output
        _write("qk_norm_rope", "norm rope prompt", 4096, 32, 8, 128, 128, 16),
        # a few tokens of a small model whose rotation covers half of each head, in pairs
        _write("qk_norm_rope", "norm rope few tokens", 37, 14, 2, 64, 32, 16, interleaved=True),
        # a packed prefill of 16384 tokens into the cache
        _write("kv_write", "write prefill", 16384, 32, 8, 128, 128, 64),
        # one decode step of 13 sequences, e5m2 codes with power-of-two scales, token-major pages
        _write("kv_write", "write 13 tokens", 13, 8, 4, 96, 96, 16, fmt="e5m2", scale="ue8m0", layout="NHD"),
        # the same step of a decode batch of 64 with norm, rotation and quantisation in one pass
        _write("qk_norm_rope_kv_write", "fused decode step", 64, 32, 8, 128, 128, 16),
        # a packed prefill: every row of q, k and v once
        _write("qk_norm_rope_kv_write", "fused prefill", 16384, 32, 8, 128, 128, 32),
        # the context of a chunked prefill: 32 ragged sequences read back
        _read("kv_read", "read contexts", 32, 4096, 32, 8, 128, 16),
        # one short context of a wide head
        _read("kv_read", "read one context", 1, 301, 8, 1, 256, 32, fmt="e5m2", layout="NHD"),
        # one user, one kv head of a sharded model: only latency counts
        _read("paged_attention", "attention one user", 1, 777, 8, 1, 128, 16),
        # an ordinary decode batch of ragged lengths, pages of 16 tokens
        _read("paged_attention", "attention batch", 32, 8192, 32, 8, 128, 16),
        # two long contexts: the cache's length has to be split over the whole GPU
        _read("paged_attention", "attention long", 2, 131071, 64, 8, 128, 64, fmt="e5m2", layout="NHD"),
        # a full server: 64 ragged contexts of up to 24000 tokens
        _read("paged_attention", "attention full", 64, 24000, 32, 8, 128, 32),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qk_norm_rope", "kv_write", "qk_norm_rope_kv_write", "kv_read", "paged_attention",
                     "paged_attention"])
    d = rng.choice([64, 80, 96, 128, 128, 128, 192, 256])
    hkv = rng.choice([1, 2, 4, 5, 8])
    hq = hkv * rng.choice([1, 2, 4, 5, 7, 8, 12, 16])
    page = rng.choice([8, 16, 24, 32, 48, 64, 128, 256])
    fmt = rng.choice(["e4m3", "e4m3", "e5m2"])
    layout = rng.choice(["HND", "NHD"])
    if op in ("kv_read", "paged_attention"):
        cap = 1 << 30 if op == "paged_attention" else 1 << 27      # cache values of k
        b = _log_int(rng, 1, 128)
        longest = _log_int(rng, 1, max(1, min(131071, cap // (b * hkv * d))))
        window = rng.choice([0, 0, 0, _log_int(rng, 1, 8192)]) if op == "paged_attention" else 0
        return {k: v for k, v in _read(op, "", b, longest, hq, hkv, d, page, fmt, layout, window).items() if k != "name"}
    t = _log_int(rng, 1, max(1, min(20000, (96 << 20) // ((hq + 2 * hkv) * d))))
    r = rng.choice([d, d, d // 2 // 16 * 16])
    c = _write(op, "", t, hq, hkv, d, r, page, fmt, rng.choice(["fp32", "ue8m0"]), layout, rng.random() < 0.3)
    return {k: v for k, v in c.items() if k != "name"}


def _lens(case):
    """Ragged lengths of the batch, the longest first: a low-discrepancy sequence over 1..longest."""
    return [max(1, case["longest"] - int(case["longest"] * ((0.6180339887498949 * i) % 1.0))) for i in range(case["b"])]


# ----------------------------------------------------------------- inputs
def _pages(x, layout):
    """The same logical [pages, heads, page, dim] tensor with token-major memory for NHD."""
    return x if layout == "HND" else x.transpose(1, 2).contiguous().transpose(1, 2)


def _cos_sin(n, r):
    """fp32 [n, r]: cosines, then sines, of position * 10000^(-2 i / r), the angles in 64 bits."""
    freq = 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    d, hq, hkv, page = case["d"], case["hq"], case["hkv"], case["page"]

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

    def codes(n):
        x = randn(n, hkv, page, d).mul_(FMAX[case["fmt"]] / 4).clamp_(-FMAX[case["fmt"]], FMAX[case["fmt"]])
        return _pages(x.to(F8[case["fmt"]]).view(torch.uint8), case["layout"])

    def scales(n):
        return (torch.randn((n, hkv, page), generator=g, device="cuda") * 0.5).exp_() * (4 / FMAX[case["fmt"]])

    s = dict(case)
    if case["op"] in ("kv_read", "paged_attention"):
        lens = _lens(case)
        need = [-(-n // page) for n in lens]
        width = max(need)
        total = sum(need)
        ids = torch.randperm(total, generator=g, device="cuda").int()
        first = torch.tensor([0] + need[:-1], device="cuda").cumsum(0)
        at = torch.arange(width, device="cuda")
        inside = at < torch.tensor(need, device="cuda")[:, None]
        s["table"] = torch.where(inside, ids[(first[:, None] + at).clamp(max=total - 1)], 0).int().contiguous()
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["k"], s["v"] = codes(total), codes(total)
        s["ks"], s["vs"] = scales(total), scales(total)
        if case["op"] == "kv_read":
            s["rows"] = sum(lens)
            s["offsets"] = torch.tensor([0] + lens, device="cuda").cumsum(0).int()
            s["ko"] = torch.empty((s["rows"], hkv, d), dtype=torch.bfloat16, device="cuda")
            s["vo"] = torch.empty_like(s["ko"])
        else:
            s["q"] = randn(case["b"], hq, d)
            s["out"] = torch.empty_like(s["q"])
        return s
    t = case["t"]
    qkv = randn(t, (hq + 2 * hkv), d)             # the projection's output; q, k and v are views of it
    # channels differ in size, as a projection's do
    qkv *= (torch.randn((hq + 2 * hkv, d), generator=g, device="cuda") * 0.5).exp_().to(torch.bfloat16)
    s["q"], s["kx"], s["vx"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    s["wq"], s["wk"] = 1 + 0.1 * randn(d), 1 + 0.1 * randn(d)
    s["cos_sin"] = _cos_sin(POSITIONS, case["r"])
    s["pos"] = torch.randint(0, POSITIONS, (t,), generator=g, device="cuda")
    s["qo"] = torch.empty((t, hq, d), dtype=torch.bfloat16, device="cuda")
    s["ko"] = torch.empty((t, hkv, d), dtype=torch.bfloat16, device="cuda")
    if case["op"] != "qk_norm_rope":
        pages = -(-t // page) + 3
        s["k"], s["v"], s["ks"], s["vs"] = codes(pages), codes(pages), scales(pages), scales(pages)
        s["slots"] = torch.randperm(pages * page, generator=g, device="cuda")[:t].contiguous()
        s["slots"][t // 2::29] = -1               # padding rows of the batch: nothing is written for them
    return s


# ------------------------------------------------------------- plain forms
def _norm_rope(x, w, s):
    """fp32 [T, H, D] of bf16 x: the head's RMS norm, then the rotation of its first r channels."""
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
    r = s["r"]
    cs = s["cos_sin"][s["pos"]][:, None, :]
    c, n = cs[..., :r // 2], cs[..., r // 2:]
    if s["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * c - b * n, b * c + a * n], -1)
    return torch.cat([y, x[..., r:]], -1)


def _quant(x, s):
    """fp32 [T, H, D] -> (codes as bytes, fp32 scale [T, H])."""
    f = FMAX[s["fmt"]]
    sc = (x.abs().amax(-1) / f).clamp(min=TINY)
    if s["scale"] == "ue8m0":
        m, e = torch.frexp(sc)                    # sc = m 2^e, m in [1/2, 1): an exact power of two has m = 1/2
        sc = torch.ldexp(torch.ones_like(sc), torch.where(m == 0.5, e - 1, e))
    return (x / sc[..., None]).clamp(-f, f).to(F8[s["fmt"]]).view(torch.uint8), sc


def _store(x, codes, scales, s):
    keep = s["slots"] >= 0
    page, row = s["slots"][keep] // s["page"], s["slots"][keep] % s["page"]
    q, sc = _quant(x[keep], s)
    codes[page, :, row] = q
    scales[page, :, row] = sc


def _cache_out(s):
    """The cache as the values its codes stand for, and the scales."""
    return {"k": s["k"].view(F8[s["fmt"]]), "v": s["v"].view(F8[s["fmt"]]), "ks": s["ks"], "vs": s["vs"]}


def _gather(codes, scales, s):
    """fp32 [B, H, L, D] of the table's pages."""
    t = s["table"].long()
    x = codes.view(F8[s["fmt"]])[t].float() * scales[t][..., None]        # [B, pages, H, P, D]
    return x.transpose(1, 2).flatten(2, 3)


def _plain(s):
    op = s["op"]
    if op == "qk_norm_rope":
        return {"q": _norm_rope(s["q"], s["wq"], s).bfloat16(), "k": _norm_rope(s["kx"], s["wk"], s).bfloat16()}
    if op == "kv_write":
        _store(s["kx"].float(), s["k"], s["ks"], s)
        _store(s["vx"].float(), s["v"], s["vs"], s)
        return _cache_out(s)
    if op == "qk_norm_rope_kv_write":
        _store(_norm_rope(s["kx"], s["wk"], s), s["k"], s["ks"], s)
        _store(s["vx"].float(), s["v"], s["vs"], s)
        return {"q": _norm_rope(s["q"], s["wq"], s).bfloat16(), **_cache_out(s)}
    at = torch.arange(s["table"].shape[1] * s["page"], device="cuda")
    lens = s["lens"][:, None]
    if op == "kv_read":
        inside = at < lens
        return {"k": _gather(s["k"], s["ks"], s).transpose(1, 2)[inside].bfloat16(),
                "v": _gather(s["v"], s["vs"], s).transpose(1, 2)[inside].bfloat16()}
    inside = at < lens
    if s["window"]:
        inside = inside & (at >= lens - s["window"])
    inside = inside[:, None, None, :]
    k, v = _gather(s["k"], s["ks"], s), _gather(s["v"], s["vs"], s)
    q = s["q"].float().view(s["b"], s["hkv"], -1, s["d"]) * (1 / math.sqrt(s["d"]))
    x = (q @ k.transpose(-1, -2)).masked_fill(~inside, -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    o = (p @ v) / p.sum(-1, keepdim=True)
    return {"out": o.flatten(1, 2).bfloat16()}


# --------------------------------------------------------- the library's calls
def _handles(s):
    """What a program keeps beside its cache: the handle of its memory, and attention's workspace."""
    import fp8_block_scaled_12_b200 as F
    if "handle" not in s and "k" in s:
        s["handle"] = F.KVCache.wrap(s["k"], s["v"], s["ks"], s["vs"], F.E4M3 if s["fmt"] == "e4m3" else F.E5M2,
                                     F.SCALE_UE8M0 if s.get("scale") == "ue8m0" else F.SCALE_FP32)
        if s["op"] == "paged_attention":
            n = F.paged_attention_ws_bytes(s["b"], s["hq"], s["handle"])
            s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return F


def _own(s):
    F = _handles(s)
    op = s["op"]
    if op == "qk_norm_rope":
        F.fp8_qk_norm_rope(s["q"], s["kx"], s["pos"], s["cos_sin"], s["qo"], s["ko"], s["wq"], s["wk"], EPS,
                           s["interleaved"])
        return {"q": s["qo"], "k": s["ko"]}
    if op == "kv_write":
        F.fp8_kv_write(s["kx"], s["vx"], s["slots"], s["handle"])
        return _cache_out(s)
    if op == "qk_norm_rope_kv_write":
        F.fp8_qk_norm_rope_kv_write(s["q"], s["kx"], s["vx"], s["pos"], s["cos_sin"], s["slots"], s["handle"], s["qo"],
                                    s["wq"], s["wk"], EPS, s["interleaved"])
        return {"q": s["qo"], **_cache_out(s)}
    if op == "kv_read":
        F.fp8_kv_read(s["handle"], s["table"], s["offsets"], s["ko"], s["vo"])
        return {"k": s["ko"], "v": s["vo"]}
    F.fp8_paged_attention(s["q"], s["handle"], s["table"], s["lens"], s["out"], s["ws"], window=s["window"])
    return {"out": s["out"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- work
def work(case):
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    if case["op"] in ("kv_read", "paged_attention"):
        lens = _lens(case)
        seen = sum(min(n, case["window"] or n) for n in lens)
        table = 4 * sum(-(-min(n, case["window"] or n) // case["page"]) for n in lens)
        cache = 2 * seen * hkv * (d + 4)
        if case["op"] == "kv_read":
            return {"bytes": cache + 2 * seen * hkv * d * 2 + table, "flops": 2 * seen * hkv * d}
        return {"bytes": cache + table + 4 * case["b"] * hq * d, "flops": 4 * seen * hq * d}
    t = case["t"]
    moved = 0
    if case["op"] != "kv_write":
        moved += t * hq * d * 4 + 8 * t + min(t, POSITIONS) * 4 * case["r"]     # q in and out, positions, their rows of the table
    moved += t * hkv * d * 4 if case["op"] == "qk_norm_rope" else 2 * t * hkv * (d * 3 + 4) + 8 * t
    heads = {"qk_norm_rope": hq + hkv, "kv_write": 2 * hkv, "qk_norm_rope_kv_write": hq + 2 * hkv}[case["op"]]
    return {"bytes": moved, "flops": t * heads * d * 8}


# ------------------------------------------------------------------ exact
def _exact_norm_rope(x, w, s):
    """The same in 64 bits, channel pair by channel pair as complex numbers."""
    x = x.double()
    x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
    r = s["r"]
    cs = s["cos_sin"].double()[s["pos"]]
    turn = torch.complex(cs[:, :r // 2], cs[:, r // 2:])[:, None]
    y = x.clone()
    first = torch.arange(r // 2, device="cuda") * (2 if s["interleaved"] else 1)
    second = first + (1 if s["interleaved"] else r // 2)
    z = torch.complex(x[..., first], x[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    d, page, f = case["d"], case["page"], FMAX[case["fmt"]]
    val = {c: s[c].view(F8[case["fmt"]]).double() for c in ("k", "v")} if case["op"].endswith("kv_write") else {}

    def put(name, x):
        live = (s["slots"] >= 0).nonzero()[:, 0]
        x, slot = x[live], s["slots"][live]
        sc = x.abs().amax(-1) / f
        if case["scale"] == "ue8m0":
            sc = torch.pow(2.0, torch.ceil(torch.log2(sc.float().double().clamp(min=TINY))))
        sc = sc.clamp(min=TINY)
        p, r = torch.div(slot, page, rounding_mode="floor"), slot % page
        val[name][p, :, r] = x / sc[..., None]
        val[name + "s"][p, :, r] = sc

    if val:
        val["ks"], val["vs"] = s["ks"].double(), s["vs"].double()
    if case["op"] == "qk_norm_rope":
        return {"q": _exact_norm_rope(s["q"], s["wq"], s), "k": _exact_norm_rope(s["kx"], s["wk"], s)}
    if case["op"] == "kv_write":
        put("k", s["kx"].double())
        put("v", s["vx"].double())
        return val
    if case["op"] == "qk_norm_rope_kv_write":
        put("k", _exact_norm_rope(s["kx"], s["wk"], s))
        put("v", s["vx"].double())
        return {"q": _exact_norm_rope(s["q"], s["wq"], s), **val}
    outs = {"k": [], "v": [], "out": []}
    table = s["table"].long()
    for i, n in enumerate(_lens(case)):
        at = torch.arange(max(0, n - case["window"]) if case["window"] else 0, n, device="cuda")
        pg, rw = table[i][at // page], at % page
        k = s["k"].view(F8[case["fmt"]])[pg, :, rw].double() * s["ks"][pg, :, rw].double()[..., None]   # [L, H, D]
        v = s["v"].view(F8[case["fmt"]])[pg, :, rw].double() * s["vs"][pg, :, rw].double()[..., None]
        if case["op"] == "kv_read":
            outs["k"].append(k)
            outs["v"].append(v)
            continue
        q = s["q"][i].double().view(case["hkv"], -1, d)
        a = torch.softmax(torch.einsum("hgd,lhd->hgl", q, k) * d ** -0.5, -1)
        outs["out"].append(torch.einsum("hgl,lhd->hgd", a, v).reshape(1, -1, d))
    return {name: torch.cat(x) for name, x in outs.items() if x}
