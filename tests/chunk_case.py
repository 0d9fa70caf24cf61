"""A batch with several new tokens a sequence over raw pages and, coded by the GPU encoder, 12-bit pages with raw
tails, with its attention in 64 bits."""
from __future__ import annotations

import math

import torch

PAGE, D = 16, 128


class ChunkCase:
    def __init__(self, seqs, hq, hkv, window=0, sinks=0, seed=0, lead=0, trail=0, k_scale=1.0, v_scale=1.0, wide=0):
        """seqs: [(new tokens, tokens with them)]; lead and trail: rows of no sequence before and behind them; wide:
        columns of the page table behind the longest sequence's."""
        import decode_attention_value_gb300 as kvz

        self.kvz, self.seqs, self.hq, self.hkv, self.G = kvz, seqs, hq, hkv, hq // hkv
        self.window, self.sinks = window, sinks
        g = torch.Generator(device="cuda").manual_seed(7000 + seed)
        dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        start = [lead]
        for n, _ in seqs:
            start.append(start[-1] + n)
        self.start, self.T = start, start[-1] + trail
        self.q_start, self.seq_lens = dev(start), dev([L for _, L in seqs])
        self.width = max([-(-L // PAGE) for _, L in seqs], default=0) + wide
        B, total = len(seqs), len(seqs) * self.width + 3
        ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        self.full_ids = ids[: B * self.width].view(B, self.width).contiguous()
        draw = lambda s: torch.randn((total, hkv, PAGE, D), generator=g, device="cuda") * s  # noqa: E731
        self.pool = torch.stack([draw(k_scale), draw(v_scale)], 2).to(torch.bfloat16)
        self.clean = self.pool.clone()
        self.q = torch.randn((self.T, hq, D), generator=g, device="cuda").to(torch.bfloat16)
        self.page_ids = self.full_ids.clone()
        for b, (n, L) in enumerate(seqs):
            if L % PAGE:  # whatever stands behind a last token is no part of the batch
                self.pool[self.full_ids[b, L // PAGE], :, :, L % PAGE:] = float("nan")
            first = max(L - n - window + 1, 0) if window else 0
            for p in range(self.width):  # pages that no new token sees are not there
                if p * PAGE >= L or (p * PAGE + PAGE <= first and p * PAGE >= sinks):
                    self.page_ids[b, p] = (-1, -7, 2 ** 31 - 1)[p % 3]
                    self.pool[self.full_ids[b, p]] = float("nan")
        self.status = kvz.new_status()
        self.coded = False

    # ---- the calls ----
    def _out(self, dtype):
        return torch.full(self.q.shape, 77.0, dtype=dtype, device="cuda")

    def run_raw(self, dtype=torch.bfloat16, out=None, **kw):
        out = self._out(dtype) if out is None else out
        self.kvz.chunk_attention_raw(self.q, self.q_start, self.page_ids, self.seq_lens, self.pool, out, self.status,
                                     window=self.window, sinks=self.sinks, **kw)
        return out

    def encode(self):
        """All pages in 12-bit form (page id = raw page id), tails in their raw pages."""
        kvz, P = self.kvz, self.pool.shape[0]
        self.meta = torch.zeros((P, self.hkv, 2), dtype=torch.int64, device="cuda")
        self.arena = torch.zeros(P * self.hkv * 2 * 4096, dtype=torch.uint8, device="cuda")
        cursors = torch.tensor([[0, self.arena.numel() // 256]], dtype=torch.int32, device="cuda")
        src = torch.randperm(P, device="cuda").to(torch.int32)
        kvz.encode_pages(self.clean, src, src, torch.zeros_like(src), self.meta, self.arena, cursors, self.status)
        self.tail_page = torch.tensor([int(self.full_ids[b, L // PAGE]) if L % PAGE else -1 for b, (_, L) in enumerate(self.seqs)],
                                      dtype=torch.int32, device="cuda")
        self.whole = self.page_ids[:, : max([L // PAGE for _, L in self.seqs], default=0)].contiguous()
        self.coded = True

    def run_coded(self, dtype=torch.bfloat16, out=None, **kw):
        if not self.coded:
            self.encode()
        out = self._out(dtype) if out is None else out
        self.kvz.chunk_attention(self.q, self.q_start, self.whole, self.seq_lens, self.tail_page, self.meta, self.arena,
                                 self.pool, out, self.status, window=self.window, sinks=self.sinks, **kw)
        return out

    # ---- 64 bits ----
    def reference(self, skip=()):
        """(output, sum of weights times |v|, error of a weight, steps) of every row in 64 bits; skip: (sequence, page)
        pairs that are left out.  A score is a sum of 128 exact products in eight fp32 steps of a 16-term sum, each off
        by at most 17 half-steps of the terms' sum a = sum |q k| / sqrt(128); a weight's relative error is twice that
        (itself and the row's maximum) and 2^-21 for the exponential."""
        out = torch.zeros(self.q.shape, dtype=torch.float64, device="cuda")
        size, rel = torch.zeros_like(out), torch.zeros(self.q.shape[:2], dtype=torch.float64, device="cuda")
        steps = 40.0
        for b, (n, L) in enumerate(self.seqs):
            if n == 0 or L == 0:
                continue
            j = torch.arange(L, device="cuda")
            p = torch.arange(L - n, L, device="cuda")
            seen = j[None] <= p[:, None]
            if self.window:
                seen &= (j[None] > p[:, None] - self.window) | (j[None] < self.sinks)
            for sb, page in skip:
                if sb == b:
                    seen &= (j // PAGE != page)[None]
            kv = self.clean[self.full_ids[b, j // PAGE].long(), :, :, j % PAGE].double()  # [L][hkv][2][128]
            rows = slice(self.start[b], self.start[b] + n)
            for h in range(self.hkv):
                q = self.q[rows, h * self.G: (h + 1) * self.G].double()
                k, v = kv[:, h, 0], kv[:, h, 1]
                s = torch.einsum("tgd,kd->tgk", q, k) / math.sqrt(D)
                a = torch.einsum("tgd,kd->tgk", q.abs(), k.abs()) / math.sqrt(D)
                s = s.masked_fill(~seen[:, None], -math.inf)
                w = torch.softmax(s, -1).nan_to_num(0.0)  # (a row that sees nothing)
                out[rows, h * self.G: (h + 1) * self.G] = w @ v
                size[rows, h * self.G: (h + 1) * self.G] = w @ v.abs()
                rel[rows, h * self.G: (h + 1) * self.G] = a.masked_fill(~seen[:, None], 0.0).amax(-1)
            steps = max(steps, L / 16 + 40.0)
        return out, size, 2 * (8 * 17 * 2.0 ** -24 * rel) + 2.0 ** -21, steps

    def check(self, got, ref=None, what=""):
        """An output is off by twice its weights' error (weights and their sum) of size = sum p |v|, by 17 * 2^-24 of it a
        step of 16 keys (and the joins' few steps), by the rounding of the weights to BF16 (2^-8 of each at most) where the
        output is BF16 and by 2^-23 where it is fp32 (three parts), and by the output's own rounding."""
        want, size, weight, steps = self.reference() if ref is None else ref
        bf16 = got.dtype is torch.bfloat16
        tol = size * (2 * weight[..., None] + 17 * 2.0 ** -24 * steps + (2.0 ** -8 if bf16 else 2.0 ** -23))
        if bf16:
            tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
        rows = torch.zeros(self.T, dtype=torch.bool, device="cuda")
        rows[self.start[0]: self.start[-1]] = True
        assert (got[~rows] == 77.0).all(), f"{what}: rows of no sequence changed"
        assert torch.isfinite(got).all(), f"{what}: not finite"
        err = (got.double() - want).abs()
        over = (err - tol)[rows]
        assert (over <= 0).all(), f"{what}: {over.max().item():.3e} over, {(over > 0).sum().item()} values"
        return (err[rows].norm() / want[rows].norm().clamp(min=1e-30)).item()
