"""The operators of an attention block run together: projection, norm, rotation and cache
write in one pass, attention over the pages, quantisation of its output and the output
projection; step after step, eagerly, in a CUDA graph, and on streams of their own."""
import pytest
import torch

import fp8_block_scaled_12_b200 as F
import synth
from _kv_ref import attention_ref, check_attention, make_cache

pytestmark = pytest.mark.gpu


class Block:
    """B sequences of ragged lengths, prefilled, with room for `room` more tokens each."""

    def __init__(self, B=5, H=2, G=4, D=128, P=16, room=20, dev="cuda", seed=0):
        self.B, self.H, self.G, self.D, self.P, self.dev = B, H, G, D, P, dev
        self.K = 256
        Hq = H * G
        g = torch.Generator(device=dev).manual_seed(seed)
        self.lens = [37 * i + 1 for i in range(B)]
        width = -(-(max(self.lens) + room) // P)
        self.cache = make_cache(B * width, P, H, D)
        self.table = torch.randperm(B * width, generator=torch.Generator().manual_seed(seed)).int().view(B, width).to(dev)
        self.cs = F.rope_table(4096, D, device=dev)
        self.wq, self.wk = ((1 + 0.1 * torch.randn(D, generator=g, device=dev)).to(torch.bfloat16) for _ in range(2))
        self.qkv_w = F.weight_quant(synth.weights((Hq + 2 * H) * D, self.K, 0.06, seed=seed, device=dev))
        self.out_w = F.weight_quant(synth.weights(self.K, Hq * D, 0.03, seed=seed + 1, device=dev))
        self.n = torch.tensor(self.lens, dtype=torch.int32, device=dev)
        # prompts, through the separate norm and write
        T = sum(self.lens)
        qkv = self.project(synth.activations(T, self.K, seed=seed, device=dev))
        pos = torch.cat([torch.arange(n) for n in self.lens]).to(dev)
        seq = torch.cat([torch.full((n,), b) for b, n in enumerate(self.lens)]).to(dev)
        q, k, v = self.split(qkv)
        _, kn = F.qk_norm_rope(q, k, pos, self.cs, self.wq, self.wk)
        F.kv_write(kn, v, self.slots(seq, pos), self.cache)

    def project(self, x):
        qa, sa = F.act_quant(x)
        return F.block_gemm(qa, sa, *self.qkv_w).view(x.shape[0], -1, self.D)

    def split(self, qkv):
        Hq = self.H * self.G
        return qkv[:, :Hq], qkv[:, Hq:Hq + self.H], qkv[:, Hq + self.H:]

    def slots(self, seq, pos):
        return self.table[seq, pos // self.P].long() * self.P + pos % self.P

    def step(self, x):
        """One token per sequence at position n; returns (rotated q, attention's output, the block's)."""
        pos = self.n.long()
        q, k, v = self.split(self.project(x))
        slots = self.slots(torch.arange(self.B, device=self.dev), pos)
        qn = F.qk_norm_rope_kv_write(q, k, v, pos, self.cs, slots, self.cache, self.wq, self.wk)
        o = F.paged_attention(qn, self.cache, self.table, (pos + 1).int())
        oa, os = F.act_quant(o.view(self.B, -1))
        return qn, o, F.block_gemm(oa, os, *self.out_w)

    def context(self):
        """The cache read back for 64-bit attention: its codes times scales."""
        kv = []
        for b, n in enumerate(self.n.tolist()):
            tok = torch.arange(n, device=self.dev)
            pg, rw = self.table[b].long()[tok // self.P], tok % self.P
            kv.append(tuple(c[pg, :, rw].view(torch.float8_e4m3fn).double() * s[pg, :, rw].double()[..., None]
                            for c, s in ((self.cache.k, self.cache.k_scale), (self.cache.v, self.cache.v_scale))))
        return kv


def test_steps(cuda_device):
    blk = Block()
    for i in range(18):                              # passes the end of a page and of a tile
        x = synth.activations(blk.B, blk.K, seed=100 + i, device="cuda")
        q, o, y = blk.step(x)
        blk.n += 1
        ref, _, tol, _ = attention_ref(q, blk.context())
        check_attention(o, ref, tol, f"step {i}")
        oa, os = F.act_quant(o.view(blk.B, -1))
        assert torch.equal(y, F.block_gemm(oa, os, *blk.out_w))
    assert F.fp8_device_error() == 0
    # the last context through the reader: what attention saw, rounded to bf16
    off = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), blk.n.cumsum(0).int()])
    k, v = F.kv_read(blk.cache, blk.table, off, int(off[-1]))
    ctx = blk.context()
    assert torch.equal(k, torch.cat([c[0] for c in ctx]).float().to(torch.bfloat16))
    assert torch.equal(v, torch.cat([c[1] for c in ctx]).float().to(torch.bfloat16))


def test_steps_in_a_graph(cuda_device):
    """Captured once, replayed with the lengths advancing on the device: the eager bits."""
    a, b = Block(seed=3), Block(seed=3)
    x = synth.activations(a.B, a.K, seed=7, device="cuda")
    snapshot = [t.clone() for t in (b.cache.k, b.cache.v, b.cache.k_scale, b.cache.v_scale)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b.step(x)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for t, o in zip((b.cache.k, b.cache.v, b.cache.k_scale, b.cache.v_scale), snapshot):
        t.copy_(o)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = b.step(x)
        b.n += 1
    for _ in range(10):
        ref = a.step(x)
        a.n += 1
        g.replay()
        torch.cuda.synchronize()
        for r, o in zip(ref, out):
            assert torch.equal(r, o)
    assert torch.equal(a.cache.k, b.cache.k) and torch.equal(a.cache.v, b.cache.v)
    assert F.fp8_device_error() == 0
    del g


def test_two_streams_at_once(cuda_device):
    """Two blocks on two streams, their calls interleaved, each with workspaces of its own."""
    blks = [Block(seed=i) for i in (5, 6)]
    refs = []
    xs = [synth.activations(b.B, b.K, seed=9, device="cuda") for b in blks]
    for b, x in zip(blks, xs):
        refs.append([t.clone() for t in b.step(x)])
    streams = [torch.cuda.Stream() for _ in blks]
    torch.cuda.synchronize()
    for _ in range(20):
        outs = []
        for b, x, s in zip(blks, xs, streams):
            with torch.cuda.stream(s):
                outs.append(b.step(x))
        torch.cuda.synchronize()
        for r, o in zip(refs, outs):
            for u, w in zip(r, o):
                assert torch.equal(u, w)
    assert F.fp8_device_error() == 0


def test_explicit_stream(cuda_device):
    """`stream=` as an object and as a handle, with another stream current."""
    blk = Block(seed=8)
    q = torch.randn((blk.B, blk.H * blk.G, blk.D), device="cuda").to(torch.bfloat16)
    ref = F.paged_attention(q, blk.cache, blk.table, blk.n)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for st in (s, s.cuda_stream):
        out = F.paged_attention(q, blk.cache, blk.table, blk.n, stream=st)
        s.synchronize()
        assert torch.equal(out, ref)


def test_workspace_and_output_are_not_read(cuda_device):
    """Whatever an earlier call (another shape, another graph) left in the workspace is harmless."""
    blk = Block(seed=9)
    q = torch.randn((blk.B, blk.H * blk.G, blk.D), device="cuda").to(torch.bfloat16)
    ref = F.paged_attention(q, blk.cache, blk.table, blk.n)
    ws = torch.empty(F.paged_attention_ws_bytes(blk.B, q.shape[1], blk.cache), dtype=torch.uint8, device="cuda")
    for fill in (0, 0xFF, 0x7F):
        ws.fill_(fill)
        out = torch.full_like(ref, float("nan"))
        F.fp8_paged_attention(q, blk.cache, blk.table, blk.n, out, ws)
        assert torch.equal(out, ref)


def test_pages_beyond_32_bit_offsets(cuda_device):
    """Write, read and attention on the last pages of a cache of 4.9 GB of k and as much of v, and
    on its first: byte offsets and elements pass 32 bits between them."""
    pages, P, H, G, D = 75000, 64, 8, 4, 128
    assert pages * P * H * D > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(3)
    for layout in ("HND", "NHD"):
        c = F.KVCache(pages, P, H, D, layout=layout)
        lens = [300, 77]
        table = torch.tensor([[pages - 1, pages - 3, 0, pages - 7, 2], [pages - 2, 1, 5, 5, 5]], dtype=torch.int32,
                             device="cuda")
        kv, slots = [], []
        for b, n in enumerate(lens):
            t = torch.arange(n, device="cuda")
            slots.append(table[b].long()[t // P] * P + t % P)
        slots = torch.cat(slots)
        k, v = (torch.randn((sum(lens), H, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        F.kv_write(k, v, slots, c)
        off = torch.tensor([0, 300, 377], dtype=torch.int32, device="cuda")
        kb, vb = F.kv_read(c, table, off, sum(lens))
        page, row = slots // P, slots % P
        k64, v64 = (x[page, :, row].view(torch.float8_e4m3fn).double() * s[page, :, row].double()[..., None]
                    for x, s in ((c.k, c.k_scale), (c.v, c.v_scale)))
        for got, want, src in ((kb, k64, k), (vb, v64, v)):
            assert torch.equal(got, want.to(torch.float32).to(torch.bfloat16))
            # a code is off by half a step of its value, 2^-4, or of the smallest step, 2^-10 of 448
            amax = src.double().abs().amax(-1, keepdim=True)
            assert ((want - src.double()).abs() <= src.double().abs() * 2 ** -4 + amax * 2 ** -10 / 448).all()
        q = torch.randn((2, H * G, D), generator=g, device="cuda").to(torch.bfloat16)
        out = F.paged_attention(q, c, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
        assert F.fp8_device_error() == 0
        ref, _, tol, _ = attention_ref(q, [(k64[:300], v64[:300]), (k64[300:], v64[300:])], None, 0)
        check_attention(out, ref, tol, "out")
        del c
