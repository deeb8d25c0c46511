"""Inputs and 64-bit references for the tests of a drafted decoding step and of cross attention."""
import math

import torch

import paged_kv_cache_149_gb300 as pa

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def starts(qlens):
    out = [0]
    for n in qlens:
        out.append(out[-1] + n)
    return out


class Paged:
    """Random K/V of each sequence in blocks of a shuffled pool; rows that hold no token are NaN."""

    def __init__(self, ctx, hkv, d, block, dtype, seed=0, spread=1.0, extra=3, num_blocks=None):
        g = torch.Generator().manual_seed(seed)
        self.ctx, self.hkv, self.d, self.block, self.dt = list(ctx), hkv, d, block, DT[dtype]
        used = [-(-max(c, 0) // block) for c in ctx]
        self.width = max(max(used, default=0), 1) + 1
        nb = num_blocks or sum(used) + extra
        self.order = torch.randperm(nb, generator=g)
        self.tables = torch.full((len(ctx), self.width), -1, dtype=torch.int32)
        at = 0
        for s, u in enumerate(used):
            self.tables[s, :u] = self.order[at:at + u].int()
            at += u
        self.k = [(torch.randn(max(c, 0), hkv, d, generator=g) * spread).to(self.dt) for c in ctx]
        self.v = [torch.randn(max(c, 0), hkv, d, generator=g).to(self.dt) for c in ctx]
        self.nb, self.g = nb, g

    def caches(self):
        kc, vc = (torch.full((self.nb, self.hkv, self.block, self.d), math.nan, dtype=self.dt) for _ in range(2))
        for s, c in enumerate(self.ctx):
            for j in range(-(-max(c, 0) // self.block)):
                a, b = j * self.block, min(c, (j + 1) * self.block)
                t = int(self.tables[s, j])
                kc[t, :, :b - a] = self.k[s][a:b].transpose(0, 1)
                vc[t, :, :b - a] = self.v[s][a:b].transpose(0, 1)
        return kc.cuda(), vc.cuda()

    def q(self, rows, hq):
        return torch.randn(rows, hq, self.d, generator=self.g).to(self.dt)


def attend64(q, k, v, scale, first=None):
    """(softmax(scale q k^T) v, sum of weights * |v|) in 64 bits; q [rows, Hq, d], k, v [c, Hkv, d];
    row i attends to keys up to first + i, or to all."""
    rows, hq, d = q.shape
    c, hkv, _ = k.shape
    if c == 0:
        z = torch.zeros(rows, hq, d, dtype=torch.float64)
        return z, z
    G = hq // hkv
    x = q.double().view(rows, hkv, G, d)
    s = torch.einsum("rhgd,thd->rhgt", x, k.double()) * scale
    if first is not None:
        late = torch.arange(c)[None, :] > first + torch.arange(rows)[:, None]
        s = s.masked_fill(late[:, None, None, :], -math.inf)
    w = torch.softmax(s, -1)
    o = torch.einsum("rhgt,thd->rhgd", w, v.double())
    a = torch.einsum("rhgt,thd->rhgd", w, v.double().abs())
    return o.reshape(rows, hq, d), a.reshape(rows, hq, d)


def half_step(dt):
    return torch.finfo(dt).eps / 2


def attention_tolerance(ref, mass, dt, d):
    """What the arithmetic allows.  Weights are rounded to dt (half a step of each: u of
    sum w |v|), outputs too (u of the value).  Scores are sums of d products in fp32, each addition off
    by 2^-23 of the partial sums' size at most, sum |q k| scale < 2 d^0.5 for values of size 1 (the
    tests' mean is 0.64 d / d^0.5): weights off by twice 2^-23 d * 2 d^0.5, exp2 and its argument by
    2^-21, sums of weights and of products by 2^-21 more."""
    u = half_step(dt)
    rel = 2 * 2.0 ** -23 * d * 2 * math.sqrt(d) + 2 * 2.0 ** -21
    return u * (mass * (1 + 4 * u) + ref.abs()) + rel * mass + torch.finfo(dt).tiny * u * 2


def run(call, p, q, qs, ctx, scale, out=None, caches=None, **kw):
    kc, vc = caches or p.caches()
    pa.get_device_error()
    out = call(q.cuda(), kc, vc, p.tables.cuda(), i32(ctx), i32(qs), scale, out=out, **kw)
    return out.cpu(), pa.get_device_error()
