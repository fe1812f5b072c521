"""Paged caches for the tests: requests with given lengths on scattered pages,
everything that no request owns filled with NaN."""
from __future__ import annotations

import numpy as np

from oracle import paged as oracle


def torch_dtype(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float16


class PagedCase:
    """``rows``: (cached tokens with the new ones, new tokens) per request."""

    def __init__(self, rows, Hq, Hk, D, page, dtype, seed=0, spare=5, extra_tokens=0, qkv=True,
                 n_pages=None, spread=1.0, device="cuda:0"):
        import torch
        g = torch.Generator().manual_seed(seed)
        self.rows, self.Hq, self.Hk, self.D, self.page, self.dtype = rows, Hq, Hk, D, page, dtype
        dt = torch_dtype(dtype)
        pages = [-(-L // page) for L, _ in rows]
        total = sum(pages) + spare if n_pages is None else n_pages
        # the highest page numbers are in use
        order = (torch.randperm(sum(pages) + spare, generator=g) + total - sum(pages) - spare).to(torch.int32)
        width = max(pages + [1]) + 1
        table = torch.full((max(len(rows), 1), width), 2 ** 31 - 1, dtype=torch.int32)[:len(rows)]
        self.k_cache = torch.full((total, Hk, page, D), float("nan"), dtype=dt, device=device)
        self.v_cache = torch.full((total, Hk, page, D), float("nan"), dtype=dt, device=device)
        self.host = []
        at, cu = 0, [0]
        for b, (L, n) in enumerate(rows):
            ids = order[at:at + pages[b]]
            at += pages[b]
            table[b, :pages[b]] = ids
            kv = (torch.randn(2, L, Hk, D, generator=g) * spread).to(dt)
            for i in range(2):
                padded = torch.full((pages[b] * page, Hk, D), float("nan"), dtype=dt)
                padded[:L] = kv[i]
                cache = self.v_cache if i else self.k_cache
                cache[ids.long().to(device)] = padded.view(pages[b], page, Hk, D).transpose(1, 2).to(device)
            self.host.append(kv.double().numpy())
            cu.append(cu[-1] + n)
        self.T = cu[-1] + extra_tokens
        heads = Hq + 2 * Hk if qkv else Hq
        self.qkv = torch.randn(self.T, heads, D, generator=g).mul(spread).to(dt).to(device)
        self.q = self.qkv[:, :Hq]
        self.block_table = table.to(device)
        self.cu_new = torch.tensor(cu, dtype=torch.int32, device=device)
        self.kv_len = torch.tensor([L for L, _ in rows], dtype=torch.int32, device=device)
        self.scale = D ** -0.5

    def run(self, **kw):
        from speculative_decoding_verification_25_gb300 import api
        return api.paged_attention(self.q, self.k_cache, self.v_cache, self.block_table, self.cu_new,
                                   self.kv_len, scale=self.scale, want_lse=True, **kw)

    def reference(self):
        """The oracle on each request's own keys and values (as one page)."""
        q = self.q.double().cpu().numpy()
        out, lse = np.zeros((self.T, self.Hq, self.D)), np.full((self.T, self.Hq), -np.inf)
        tol, lse_tol = np.zeros_like(out), np.zeros_like(lse)
        at = 0
        for (L, n), kv in zip(self.rows, self.host):
            if L and n:
                r = oracle.attention(q[at:at + n], kv[0].transpose(1, 0, 2)[None], kv[1].transpose(1, 0, 2)[None],
                                     np.zeros((1, 1), int), [0, n], [L], self.scale, self.dtype)
                out[at:at + n], lse[at:at + n] = r.out, r.lse
                tol[at:at + n], lse_tol[at:at + n] = r.out_tol, r.lse_tol
            at += n
        return oracle.Attention(out, lse, tol, lse_tol)

    def check(self, result):
        ref = self.reference()
        out, lse = result.out.double().cpu().numpy(), result.lse.double().cpu().numpy()
        np.testing.assert_array_equal(np.isneginf(lse), np.isneginf(ref.lse))
        assert np.isfinite(out).all()
        off = np.abs(out - ref.out) - ref.out_tol
        assert (off <= 0).all(), f"out is {off.max():.3g} past its bound at {np.unravel_index(off.argmax(), off.shape)}"
        fine = np.isfinite(ref.lse)
        off = np.abs(lse[fine] - ref.lse[fine]) - ref.lse_tol[fine]
        assert (off <= 0).all(), f"lse is {off.max():.3g} past its bound"
