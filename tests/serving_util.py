"""Helpers of the paged-cache tests: caches on the GPU in several layouts, and the
same cache as the oracle's arrays."""
from __future__ import annotations

import numpy as np
import torch

import roofline_driven_optimisation_gb300 as g

KV_DTYPE = {g.KV_E4M3: torch.float8_e4m3fn, g.KV_INT8: torch.int8}


class Case:
    """A cache with random contents: every code of the pool (NaN codes among them in
    E4M3) and every scale, so that what a call must not use is there to be found."""

    def __init__(self, fmt, heads, dim, page, lengths, new=0, layout="pages_heads", spare=3, seed=0, offset=0,
                 extra=0):
        rng = self.rng = np.random.default_rng(seed)
        self.fmt, self.heads, self.dim, self.page = fmt, heads, dim, page
        need = [-(-(n + new) // page) for n in lengths]
        cols = max(1, max(need, default=0))
        self.pages = sum(need) + spare
        order = rng.permutation(self.pages)
        table = rng.integers(-7, 9999, (len(lengths), cols))       # unused columns hold anything
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.used = order[:at]
        self.np = {"table": table}
        width = dim + extra
        shape = {"pages_heads": (self.pages, heads, page, width), "pages_tokens": (self.pages, page, heads, width),
                 "heads_pages": (heads, self.pages, page, width)}[layout]
        perm = {"pages_heads": (0, 1, 2, 3), "pages_tokens": (0, 2, 1, 3), "heads_pages": (1, 0, 2, 3)}[layout]
        self.flat, self.views = {}, {}
        for name in ("k", "v"):
            codes = rng.integers(0, 256, shape).astype(np.uint8)
            s = rng.uniform(0.002, 0.02, (self.pages, heads)).astype(np.float32)
            flat = torch.zeros(codes.size + 64, dtype=torch.uint8)
            flat[offset:offset + codes.size] = torch.from_numpy(codes.reshape(-1))
            flat = flat.cuda()
            self.flat[name] = flat
            view = flat[offset:offset + codes.size].view(shape)[..., :dim].permute(perm)
            self.views[name] = view.view(KV_DTYPE[fmt])
            self.np[name] = view.cpu().numpy().copy()
            self.np[name + "s"] = s
            self.views[name + "s"] = torch.from_numpy(s).cuda()
        # read contents are finite: NaN codes become 0 where a sequence's tokens are
        if fmt == g.KV_E4M3:
            for b, n in enumerate(lengths):
                for t in range(n):
                    p, r = table[b, t // page], t % page
                    for name in ("k", "v"):
                        c = self.np[name][p, :, r]
                        c[(c & 0x7F) == 0x7F] = 0
            self.put()
        self.table = torch.from_numpy(table.astype(np.int32)).cuda()
        self.cache = g.KVCache(self.views["k"], self.views["v"], self.views["ks"], self.views["vs"], self.table)

    def put(self):
        for name in ("k", "v"):
            self.views[name].view(torch.uint8).copy_(torch.from_numpy(self.np[name]))
            self.views[name + "s"].copy_(torch.from_numpy(self.np[name + "s"]))

    def got(self, name):
        t = self.views[name]
        return (t if name.endswith("s") else t.view(torch.uint8)).cpu().numpy()


def check_status():
    torch.cuda.synchronize()
    status, where = g.device_status()
    assert status == 0, f"device status {status} at site {where}"
