"""A loop of decoding steps with drafts, as a server runs it: positions and cache write, attention,
verdict, blocks given back -- over the host pool, and as one captured graph."""
import math

import numpy as np
import torch

import pytest

import paged_kv_cache_149_gb300 as pa
from drafts_harness import attend64, attention_tolerance, i32, starts
from test_gpu_rotary import angles64, close, turned64

pytestmark = pytest.mark.gpu

HQ, HKV, D, B, V = 4, 2, 64, 16, 97
SCALE = 1 / math.sqrt(D)


class Model:
    """Rows of q, k and v from the token alone, and probabilities from the attention's output."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        self.table = torch.randn(V, (HQ + 2 * HKV) * D, generator=g).bfloat16().cuda()
        self.head = (0.5 * torch.randn(HQ * D, V, generator=g)).cuda()

    def qkv(self, tokens):
        q, k, v = self.table[tokens.long()].split([HQ * D, HKV * D, HKV * D], 1)
        return q.unflatten(1, (HQ, D)), k.unflatten(1, (HKV, D)), v.unflatten(1, (HKV, D))

    def probs(self, out):
        return torch.softmax(out.float().flatten(1) @ self.head, -1)


def test_steps_over_the_host_pool():
    m = Model(1)
    rng = np.random.default_rng(3)
    gen = torch.Generator(device="cuda").manual_seed(5)
    pool = pa.BlockPool(64, B, rng.permutation(64).astype(np.int32))
    kc, vc = (torch.full((64, HKV, B, D), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    freqs, amp = pa.rotary_frequencies(D)
    f = angles64(D, 10000.0)
    work = pa.make_split_workspace(HQ, HKV, D)
    n = 3
    history = [list(rng.integers(0, V, k)) for k in (5, 33, 16)]  # tokens known; the last is not cached yet
    for s in range(n):
        pool.allocate(s, 0)
    pa.get_device_error()
    accepted = 0
    for step in range(8):
        # a prompt first, then the last token and up to four drafts
        if step == 0:
            fed = [list(h) for h in history]
        else:
            fed = [[h[-1]] + list(rng.integers(0, V, rng.integers(0, 5))) for h in history]
        rows = [len(x) for x in fed]
        qs = starts(rows)
        for s in range(n):
            for _ in range(rows[s]):
                _, cow = pool.append_slot(s)
                assert cow is None
        ctx = [pool.context_len(s) for s in range(n)]
        width = max(len(pool.block_table(s)) for s in range(n)) + 1
        tables = np.full((n, width), -1, np.int32)
        for s in range(n):
            t = pool.block_table(s)
            tables[s, :len(t)] = t
        tables = torch.from_numpy(tables).cuda()
        tokens = i32([x for y in fed for x in y] + [0, 0])  # a padded batch
        q, k, v = m.qkv(tokens)
        dctx, dqs = i32(ctx), i32(qs)
        turned = pa.rotary_append(q, k, v, kc, vc, tables, dctx, dqs, freqs, amplitude=amp)
        if step == 0:  # the prompt: the same rows by the prefill
            out = torch.zeros_like(turned)
            pa.prefill(turned, kc, vc, tables, dctx, dqs, SCALE, max(rows), out=out)
        else:
            out = torch.zeros_like(turned)
            pa.decode_drafts(turned, kc, vc, tables, dctx, dqs, SCALE, out=out, workspace=work)
        p = m.probs(out)
        d = torch.softmax(torch.log(p) + 0.3 * torch.randn(p.shape, generator=gen, device="cuda"), -1)
        if step > 0:
            # drafts that the draft model might have proposed after the rows before them
            for s in range(n):
                for i in range(qs[s], qs[s + 1] - 1):
                    assert tokens[i + 1] == fed[s][i + 1 - qs[s]]
            u = 0.3 * torch.rand(len(tokens), generator=gen, device="cuda")
            got, emitted, left = pa.verify_drafts(tokens, p, d, u, dqs, dctx)
        else:
            # the prompt's last row alone is asked for a token: no drafts
            last = dqs[1:].long() - 1
            got, emitted, left = pa.verify_drafts(tokens[last], p[last].contiguous(), None,
                                                  torch.rand(n, generator=gen, device="cuda"),
                                                  i32([0, 1, 2, 3]), dctx)
        assert pa.get_device_error() == 0
        cache_k, cache_v, host = kc.cpu(), vc.cpu(), tables.cpu()
        out, turned = out.cpu(), turned.cpu()
        for s in range(n):
            # what the attention saw: the history without its last token, then what was fed
            seen = (history[s][:-1] if step else []) + fed[s]
            assert len(seen) == ctx[s]
            pos = torch.arange(ctx[s])
            kk, vv = (c[host[s, pos // B].long(), :, pos % B] for c in (cache_k, cache_v))
            _, k0, v0 = m.qkv(torch.tensor(seen, dtype=torch.int32, device="cuda"))
            close(kk, *turned64(k0.cpu(), pos, f, False, amp), kk.dtype)
            assert torch.equal(vv, v0.cpu())
            a, b = qs[s], qs[s + 1]
            ref, mass = attend64(turned[a:b], kk, vv, SCALE, ctx[s] - (b - a))
            assert ((out[a:b].double() - ref).abs() <= attention_tolerance(ref, mass, kk.dtype, D)).all()
            e = int(emitted[s])
            new = got[s:s + 1].tolist() if step == 0 else got[a:a + e].tolist()
            assert e >= 1 and new[:-1] == fed[s][1:e] if step else e == 1
            accepted += e - 1
            history[s] += new
            keep = ctx[s] - (0 if step == 0 else b - a - e)
            assert step == 0 or int(left[s]) == keep
            pool.truncate(s, keep)
            assert keep == len(history[s]) - 1 and len(pool.block_table(s)) == -(-keep // B)
    assert accepted > 0
    assert (out[0] != 0).any()
    used = sum(len(pool.block_table(s)) for s in range(n))
    assert pool.num_free() == 64 - used


def test_a_captured_step_repeats_on_the_gpu():
    """The whole step as one graph: lengths go from step to step in device memory; each replay is
    checked against the calls made one by one on a copy."""
    m = Model(2)
    gen = torch.Generator(device="cuda").manual_seed(7)
    n, k = 4, 4  # every sequence feeds its last token and three drafts
    freqs, amp = pa.rotary_frequencies(D)
    past = [3, 40, 100, 16]
    width = 16
    tables = torch.randperm(n * width, generator=torch.Generator().manual_seed(1)).int().view(n, width).cuda()
    qs = i32([k * s for s in range(n + 1)])

    def fresh():
        g = torch.Generator(device="cuda").manual_seed(9)
        st = dict(ctx=i32([p + k for p in past]), tokens=torch.zeros(n * k, dtype=torch.int32, device="cuda"),
                  u=torch.zeros(n * k, device="cuda"), left=i32([0] * n), emitted=i32([0] * n),
                  out=torch.zeros(n * k, dtype=torch.int32, device="cuda"),
                  kc=torch.randn(n * width, HKV, B, D, generator=g, device="cuda").bfloat16(),
                  vc=torch.randn(n * width, HKV, B, D, generator=g, device="cuda").bfloat16(),
                  work=pa.make_split_workspace(HQ, HKV, D))
        return st

    def step(st):
        q, kk, vv = m.qkv(st["tokens"])
        t = pa.rotary_append(q, kk, vv, st["kc"], st["vc"], tables, st["ctx"], qs, freqs, amplitude=amp)
        o = pa.decode_drafts(t, st["kc"], st["vc"], tables, st["ctx"], qs, SCALE, workspace=st["work"])
        pa.verify_drafts(st["tokens"], m.probs(o), None, st["u"], qs, st["ctx"], out=st["out"], emitted=st["emitted"],
                         context_next=st["left"])
        torch.add(st["left"], k, out=st["ctx"])
        return o

    a, b = fresh(), fresh()
    step(a)  # (what loads kernels and libraries comes before the capture)
    a = fresh()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        oa = step(a)
    a_, = [fresh()]
    for key in ("ctx", "kc", "vc"):
        a[key].copy_(a_[key])
    for _ in range(12):
        tokens = torch.randint(0, V, (n * k,), generator=gen, device="cuda").int()
        u = 0.02 * torch.rand(n * k, generator=gen, device="cuda")
        for st in (a, b):
            st["tokens"].copy_(tokens)
            st["u"].copy_(u)
        graph.replay()
        ob = step(b)
        torch.cuda.synchronize()
        assert torch.equal(oa, ob)
        for key in ("out", "emitted", "left", "ctx", "kc", "vc"):
            assert torch.equal(a[key], b[key]), key
    assert pa.get_device_error() == 0
    assert (a["ctx"] > i32([p + k for p in past])).all()
