"""Sequences in a cache of their own for the attention tests, with the values as the cache stores them in 64 bits.

The pool is filled with NaN first, so that a read of a slot that no token owns shows."""
import numpy as np
import torch

import compress_ref
import paged_kv_cache_134_gb300 as P

MODEL = {"f16": torch.float16, "bf16": torch.bfloat16}


class Setup:
    def __init__(self, lens, hq=4, hkv=4, d=128, bs=16, kv="f16", model="f16", seed=0, width=0, extra=5):
        self.lens, self.hq, self.hkv, self.d, self.bs, self.kv, self.model = list(lens), hq, hkv, d, bs, kv, model
        g = torch.Generator().manual_seed(seed)
        need = [(n + bs - 1) // bs for n in self.lens]
        total = sum(need)
        self.nb = total + extra
        order = torch.randperm(self.nb, generator=g)[:total].to(torch.int32)
        t = torch.full((len(self.lens), max(1, width, *need)), -1, dtype=torch.int32)
        at = 0
        for i, n in enumerate(need):
            t[i, :n] = order[at:at + n]
            at += n
        n = sum(self.lens)
        md = MODEL[model]
        k, v = (torch.randn(n, hkv, d, generator=g).to(md) for _ in range(2))
        seq = torch.repeat_interleave(torch.arange(len(self.lens)), torch.tensor(self.lens, dtype=torch.long))
        pos = torch.cat([torch.arange(m) for m in self.lens] + [torch.zeros(0, dtype=torch.long)])
        self.slots = (t[seq, pos // bs].long() * bs + pos % bs).cuda() if n else torch.zeros(0, dtype=torch.long).cuda()
        self.tables, self.context = t.cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda()
        self.cache = P.KVCache(self.nb, bs, hkv, d, kv_dtype=kv, model_dtype=model)
        self.cache.view()[0].fill_(255)
        if kv == "fp8":
            s = [(x.float().abs().amax(dim=(0, 2)) / 448).clamp(min=1e-6) if n else torch.ones(hkv) for x in (k, v)]
            self.scales = tuple(x.cuda() for x in s)
            self.cache.set_scales(*self.scales)
            codes = [(x.float() / f[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn) for x, f in zip((k, v), s)]
            self.k64, self.v64 = ((c.double() * f[:, None].double()).numpy() for c, f in zip(codes, s))
        else:
            self.k64, self.v64 = k.double().numpy(), v.double().numpy()
        if kv == "int4" and n:
            rows = [compress_ref.quantise4(x, model) for x in (self.k64, self.v64)]
            self.k64, self.v64 = (compress_ref.values4(*r) for r in rows)
            self.steps = tuple(float(r[1].max()) for r in rows)
        self.given = k.cuda(), v.cuda()
        if n:
            P.paged_kv_append(self.cache, *self.given, self.slots)
        self.at = np.concatenate([[0], np.cumsum(self.lens)])
        self.gen = g

    def rows(self, i):
        """(k, v) of sequence i, [L, Hkv, D] float64."""
        s = slice(self.at[i], self.at[i + 1])
        return self.k64[s], self.v64[s]

    def queries(self, n):
        q = torch.randn(n, self.hq, self.d, generator=self.gen).to(MODEL[self.model])
        return q.cuda(), q.double().numpy()

    def spoil(self, i, positions):
        """NaN and infinities where the tokens at these positions of sequence i are stored."""
        if not len(positions):
            return
        slots = self.slots[self.at[i] + torch.as_tensor(np.asarray(positions)).long().cuda()]
        if self.kv == "int4":  # steps and offsets NaN
            row = torch.full((len(slots), self.hkv, self.d), float("nan"), dtype=MODEL[self.model], device="cuda")
            P.paged_kv_append(self.cache, row, row, slots)
            return
        if self.kv == "fp8":
            pool = self.cache.view()[0].view(self.nb, 2, self.hkv, self.bs, self.d)
            pool[slots // self.bs, :, :, slots % self.bs] = 0x7F
            return
        pool = self.cache.view()[0].view(MODEL[self.model]).view(self.nb, 2, self.hkv, self.bs, self.d)
        bad = torch.full((len(slots), 2, self.hkv, self.d), float("nan"), device="cuda")
        bad[..., ::3], bad[..., 1::3] = float("inf"), -float("inf")
        pool[slots // self.bs, :, :, slots % self.bs] = bad.to(pool.dtype)
