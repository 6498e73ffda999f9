"""Child process of test_failure_attention.py: the paged attention with its waits limited to
1 ns, so every CTA gives up at its first wait that does not succeed at once, drains what it has
issued and returns; then the same calls at the normal limit, which give their earlier bits.  The
workspace starts as garbage, so the join sees entries that were never written.  Prints OK."""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_scaled_12_b200 as F  # noqa: E402

TIMEOUT = 6


def main():
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    g = torch.Generator(device=dev).manual_seed(1)
    cases = {}
    for name, B, Hq, H, D, P, L in (("8 heads", 5, 8, 1, 128, 16, 3000), ("16 heads", 2, 32, 2, 64, 32, 9000),
                                    ("wide", 3, 8, 2, 256, 64, 2000)):
        width = -(-L // P)
        c = F.KVCache(B * width, P, H, D)
        for t in (c.k, c.v):
            t.copy_(torch.randint(0, 124, t.shape, generator=g, device=dev).to(torch.uint8))
        c.k_scale.fill_(1e-3)
        c.v_scale.fill_(1e-2)
        table = torch.arange(B * width, dtype=torch.int32, device=dev).view(B, width)
        lens = torch.tensor([max(0, L - 700 * b) for b in range(B)], dtype=torch.int32, device=dev)
        q = torch.randn((B, Hq, D), generator=g, device=dev).to(torch.bfloat16)
        out = torch.empty_like(q)
        ws = torch.full((F.paged_attention_ws_bytes(B, Hq, c),), 0x7F, dtype=torch.uint8, device=dev)
        cases[name] = (lambda a=(q, c, table, lens, out, ws): F.fp8_paged_attention(*a), out, ws)
    ref = {}
    for name, (fn, out, _) in cases.items():
        fn()
        assert F.fp8_device_error() == 0, name
        ref[name] = out.clone()
    F.fp8_set_wait_limit_ns(1)
    try:
        for fill in (0x7F, 0x00, 0x3C):
            for name, (fn, out, ws) in cases.items():
                ws.fill_(fill)
                fn()
                status = F.fp8_device_error()
                assert status == TIMEOUT, f"{name}: status {status} with a 1 ns wait limit"
    finally:
        F.fp8_set_wait_limit_ns(0)
    for name, (fn, out, _) in cases.items():
        out.zero_()
        fn()
        assert F.fp8_device_error() == 0, name
        assert torch.equal(out, ref[name]), f"{name}: output changed after abort"
    print("OK")


if __name__ == "__main__":
    main()
