"""4-bit caches for the tests: those of PagedCase, encoded by the oracle.  What
no request owns has NaN for its scales and any codes."""
from __future__ import annotations

import numpy as np

from oracle import paged_fp4 as oracle
from oracle.paged import Attention
from paged_util import PagedCase


class Fp4Case(PagedCase):
    def __init__(self, rows, Hq, Hk, D, page, dtype, seed=0, gains=(1.0, 1.0), **kw):
        super().__init__(rows, Hq, Hk, D, page, dtype, seed, **kw)
        self.gains = gains
        self.encode()

    def encode(self):
        """The cache and the requests' values anew, from the 16-bit ones."""
        import torch
        from speculative_decoding_verification_25_gb300 import api
        parts = []
        rng = np.random.default_rng(1)
        for cache, gain in zip((self.k_cache, self.v_cache), self.gains):
            codes, scales = oracle.encode(cache.double().cpu().numpy(), gain)
            free = np.repeat(scales == oracle.NAN_SCALE, 8, -1)
            codes = np.where(free, rng.integers(0, 256, codes.shape), codes).astype(np.uint8)
            parts += [torch.from_numpy(codes).to(cache.device),
                      torch.from_numpy(scales).to(cache.device).view(torch.float8_e4m3fn)]
        self.cache = api.PagedCacheFp4(*parts)
        self.host = [np.stack([oracle.decode(*oracle.encode(kv[i], self.gains[i]), self.gains[i]) for i in range(2)])
                     for kv in self.host]

    def run(self, **kw):
        from speculative_decoding_verification_25_gb300 import api
        return api.paged_attention_fp4(self.q, self.cache, self.block_table, self.cu_new, self.kv_len, scale=self.scale,
                                       k_gain=self.gains[0], v_gain=self.gains[1], want_lse=True, **kw)

    def reference(self):
        q = self.q.double().cpu().numpy()
        out, lse = np.zeros((self.T, self.Hq, self.D)), np.full((self.T, self.Hq), -np.inf)
        tol, lse_tol = np.zeros_like(out), np.zeros_like(lse)
        at = 0
        for (L, n), kv in zip(self.rows, self.host):
            if L and n:
                r = oracle.attention(q[at:at + n], kv[0].transpose(1, 0, 2)[None], kv[1].transpose(1, 0, 2)[None],
                                     [0, n], [L], self.scale, self.dtype)
                out[at:at + n], lse[at:at + n] = r.out, r.lse
                tol[at:at + n], lse_tol[at:at + n] = r.out_tol, r.lse_tol
            at += n
        return Attention(out, lse, tol, lse_tol)
