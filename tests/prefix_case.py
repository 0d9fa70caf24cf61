"""A batch whose sequences share prefixes, as raw pages and, coded by the GPU encoder, as
12-bit pages with raw tails, with its attention in 64 bits."""
from __future__ import annotations

import math

import torch

PAGE, D = 16, 128


class PrefixCase:
    wide = False  # prefix tables too wide for the kernel that reads short prefixes with the own tokens

    def __init__(self, groups, own, hq, hkv, seed=0, lead=0, k_scale=1.0, v_scale=1.0, k=None, v=None):
        """groups: [(sequences, prefix tokens)]; own: own tokens of each sequence (lead
        sequences of no group first, then the groups', then the rest without one).  k, v:
        functions of (rows, heads, generator) giving token values, normal ones when None."""
        import decode_attention_value_gb300 as kvz

        self.kvz, self.hq, self.hkv, self.G = kvz, hq, hkv, hq // hkv
        self.groups, self.own, self.lead, B = groups, list(own), lead, len(own)
        g = torch.Generator(device="cuda").manual_seed(1000 + seed)
        self.B = B
        ends = [lead]
        for n, _ in groups:
            ends.append(ends[-1] + n)
        assert ends[-1] <= B
        dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.group_start, self.prefix_lens, self.seq_lens = dev(ends), dev([p for _, p in groups]), dev(self.own)
        pages = lambda n: (n + PAGE - 1) // PAGE  # noqa: E731
        self.pw = max([pages(p) for _, p in groups], default=0)
        self.ow = max([pages(n) for n in self.own], default=0)
        n_prefix = len(groups) * self.pw
        total = n_prefix + B * self.ow + 3
        ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        self.prefix_ids = ids[: len(groups) * self.pw].view(len(groups), self.pw).contiguous()
        if self.wide and self.pw < 130:
            pad = torch.full((len(groups), 130 - self.pw), -1, dtype=torch.int32, device="cuda")
            self.prefix_ids = torch.cat([self.prefix_ids, pad], 1)
        self.page_ids = ids[n_prefix:][: B * self.ow].view(B, self.ow).contiguous()
        draw = lambda f, scale: (torch.randn((total, hkv, PAGE, D), generator=g, device="cuda") * scale if f is None  # noqa: E731
                                 else f((total, hkv, PAGE, D), g))
        self.pool = torch.stack([draw(k, k_scale), draw(v, v_scale)], 2).to(torch.bfloat16)
        self.q = torch.randn((B, hq, D), generator=g, device="cuda").to(torch.bfloat16)
        self.pw = self.prefix_ids.shape[1]
        # whatever stands behind a last token is no part of the batch
        for ids_, lens in ((self.prefix_ids, [p for _, p in groups]), (self.page_ids, self.own)):
            for r, n in enumerate(lens):
                if n % PAGE:
                    self.pool[ids_[r, n // PAGE], :, :, n % PAGE:] = float("nan")
        self.status = kvz.new_status()
        self.coded = None

    # ---- the calls ----
    def run_raw(self, out=None, dtype=torch.float32, **kw):
        out = torch.full(self.q.shape, float("nan"), dtype=dtype, device="cuda") if out is None else out
        self.kvz.prefix_attention_raw(self.q, self.group_start, self.prefix_ids, self.prefix_lens, self.page_ids,
                                      self.seq_lens, self.pool, out, self.status, **kw)
        return out

    def encode(self):
        """All pages in 12-bit form (page id = raw page id), tails in their raw pages."""
        kvz, P = self.kvz, self.pool.shape[0]
        self.meta = torch.zeros((P, self.hkv, 2), dtype=torch.int64, device="cuda")
        self.arena = torch.zeros(P * self.hkv * 2 * 4096, dtype=torch.uint8, device="cuda")
        cursors = torch.tensor([[0, self.arena.numel() // 256]], dtype=torch.int32, device="cuda")
        src = torch.randperm(P, device="cuda").to(torch.int32)
        kvz.encode_pages(self.pool, src, src, torch.zeros_like(src), self.meta, self.arena, cursors, self.status)
        rest = lambda lens, ids: torch.tensor(  # noqa: E731
            [int(ids[r, n // PAGE]) if n % PAGE else -1 for r, n in enumerate(lens)], dtype=torch.int32, device="cuda")
        self.prefix_tail = rest([p for _, p in self.groups], self.prefix_ids)
        self.tail_page = rest(self.own, self.page_ids)
        whole = max([p // PAGE for _, p in self.groups], default=0)
        self.prefix_whole = self.prefix_ids[:, : max(whole, 130 if self.wide else 0)].contiguous()
        self.own_whole = self.page_ids[:, : max(self.own, default=0) // PAGE].contiguous()
        self.coded = True

    def run_coded(self, out=None, dtype=torch.float32, **kw):
        if not self.coded:
            self.encode()
        out = torch.full(self.q.shape, float("nan"), dtype=dtype, device="cuda") if out is None else out
        self.kvz.prefix_attention(self.q, self.group_start, self.prefix_whole, self.prefix_lens, self.prefix_tail,
                                  self.own_whole, self.seq_lens, self.tail_page, self.meta, self.arena, self.pool, out,
                                  self.status, **kw)
        return out

    # ---- 64 bits ----
    def tokens(self, ids, n, skip=()):
        """K and V [hkv][tokens][128] of a table row's n tokens, without the pages in skip."""
        t = torch.arange(n, device="cuda")
        for p in skip:
            t = t[t // PAGE != p]
        x = self.pool[ids[t // PAGE].long(), :, :, t % PAGE].double()  # [tokens][hkv][2][128]
        return x[:, :, 0].transpose(0, 1), x[:, :, 1].transpose(0, 1)

    def reference(self, skip_prefix=(), prefix=True):
        """(output, bound) in 64 bits.  The bound of a float32 output's error: a score is a sum
        of 128 exact products in eight fp32 steps of a 16-term sum, each off by at most 17
        half-steps of the terms' sum a = sum |q k| / sqrt(128); a weight's relative error is
        twice that (itself and the row's maximum), 2^-21 for the exponential and 2^-16 for its
        two BF16 parts; the output is off by twice that (weights and their sum) of sum p |v|,
        and by 17 * 2^-24 of it a step of 16 tokens, and the merges add a few steps of 2^-24."""
        out = torch.zeros(self.q.shape, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(out)
        group_of = {}
        for i, (a, b) in enumerate(zip(self.group_start.tolist(), self.group_start.tolist()[1:])):
            for s in range(a, b):
                group_of[s] = i
        shared = [self.tokens(self.prefix_ids[i], p, skip_prefix) if prefix else None
                  for i, (_, p) in enumerate(self.groups)]
        for b in range(self.B):
            k, v = self.tokens(self.page_ids[b], self.own[b])
            if b in group_of and shared[group_of[b]] is not None:
                pk, pv = shared[group_of[b]]
                k, v = torch.cat([pk, k], 1), torch.cat([pv, v], 1)
            if k.shape[1] == 0:
                continue
            q = self.q[b].double().view(self.hkv, self.G, D)
            s = q @ k.mT / math.sqrt(D)
            a = (q.abs() @ k.abs().mT / math.sqrt(D)).amax(-1)[..., None]
            p = torch.softmax(s, -1)
            size = p @ v.abs()
            steps = k.shape[1] / 16 + 40
            out[b] = (p @ v).flatten(0, 1)
            weight = 2 * (8 * 17 * 2.0 ** -24 * a) + 2.0 ** -21 + 2.0 ** -16
            tol[b] = (size * (2 * weight + 17 * 2.0 ** -24 * steps)).flatten(0, 1)
        return out, tol

    def check(self, got, ref=None, what=""):
        want, tol = self.reference() if ref is None else ref
        if got.dtype is torch.bfloat16:
            tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
        err = (got.double() - want).abs()
        assert torch.isfinite(got).all(), f"{what}: not finite"
        assert (err <= tol).all(), f"{what}: {((err - tol) / (want.abs() + 1e-3)).max().item():.3e} over"
        return (err.norm() / want.norm().clamp(min=1e-30)).item()
