"""rotary and rotary_append against rotations in 64 bits."""
import math

import pytest
import torch

import paged_kv_cache_149_gb300 as pa
from drafts_harness import DT, half_step, i32, starts

pytestmark = pytest.mark.gpu


def angles64(rd, base):
    return torch.tensor([base ** (-2.0 * i / rd) for i in range(rd // 2)], dtype=torch.float64)


def turned64(x, pos, f, interleaved, amplitude):
    """(values, |a| + |b| of each) of x [rows, heads, d] at positions pos, in 64 bits."""
    rd = 2 * len(f)
    x = x.double()
    t = pos.double()[:, None] * f
    c, s = (torch.cos(t) * amplitude)[:, None], (torch.sin(t) * amplitude)[:, None]
    out, size = x.clone(), torch.zeros_like(x)
    ia = torch.arange(0, rd, 2) if interleaved else torch.arange(rd // 2)
    ib = ia + 1 if interleaved else ia + rd // 2
    a, b = x[..., ia], x[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = (a.abs() + b.abs()) * amplitude
    return out, size


def close(got, ref, size, dt):
    # the angle in fp32 half turns is off by pi 2^-24, sincospif by 2^-22, products and sum by 2^-23 of |a| +
    # |b|: under 2^-20 of it; the output by half a step, or half the smallest value
    tol = half_step(dt) * ref.abs() + 2.0 ** -20 * size + torch.finfo(dt).smallest_normal * half_step(dt)
    assert ((got.double() - ref).abs() <= tol).all()


class Batch:
    def __init__(self, rows, past, hq, hkv, d, block, dtype, fused, extra=4, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.rows, self.past, self.dt = rows, past, DT[dtype]
        self.ctx = [r + p for r, p in zip(rows, past)]
        self.qs = starts(rows)
        self.n = self.qs[-1]
        N = self.n + extra
        x = torch.randn(N, (hq + 2 * hkv) * d, generator=g).to(self.dt).cuda()
        q, k, v = x.split([hq * d, hkv * d, hkv * d], 1)
        self.q, self.k, self.v = q.unflatten(1, (hq, d)), k.unflatten(1, (hkv, d)), v.unflatten(1, (hkv, d))
        if not fused:
            self.q, self.k, self.v = self.q.contiguous(), self.k.contiguous(), self.v.contiguous()
        used = [-(-c // block) for c in self.ctx]
        self.block = block
        first = [p // block for p in past]
        nb = sum(u - f for u, f in zip(used, first)) + 2
        order = torch.randperm(nb, generator=g).int()
        self.tables = torch.full((len(rows), max(used) + 1), -1, dtype=torch.int32)
        at = 0
        for s, (f, u) in enumerate(zip(first, used)):
            self.tables[s, f:u] = order[at:at + u - f]
            at += u - f
        self.kc = torch.randn(nb, hkv, block, d, generator=g).to(self.dt).cuda()
        self.vc = torch.randn(nb, hkv, block, d, generator=g).to(self.dt).cuda()
        self.pos = torch.cat([torch.arange(p, p + r) for r, p in zip(rows, past)])

    def slots(self):
        s = torch.repeat_interleave(torch.arange(len(self.rows)), torch.tensor(self.rows))
        return self.tables[s, self.pos // self.block].long(), self.pos % self.block


CASES = [  # dtype, d, block, hq, hkv, rotary_dim, interleaved, fused
    ("bf16", 128, 16, 32, 8, 128, False, True), ("fp16", 64, 8, 3, 1, 64, True, False),
    ("bf16", 128, 32, 5, 5, 48, False, True), ("fp16", 128, 16, 8, 2, 16, True, True),
    ("bf16", 64, 16, 16, 2, 32, False, False), ("fp16", 64, 32, 1, 1, 48, True, True),
    ("bf16", 128, 8, 64, 16, 112, True, False), ("fp16", 128, 16, 7, 7, 128, False, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_against_64_bits(case):
    dtype, d, block, hq, hkv, rd, pairs, fused = case
    # single tokens, chunks that begin inside a block, an empty sequence, positions up to millions
    b = Batch([1, 1, 0, 37, 5, 3, 2, 100], [0, 15, 3, 13, 1000, 99999, 4000001, 0], hq, hkv, d, block, dtype, fused)
    f = angles64(rd, 10000.0)
    freqs, amp = pa.rotary_frequencies(rd, 10000.0)
    assert amp == 1.0
    kc, vc = b.kc.clone(), b.vc.clone()
    pa.get_device_error()
    amp = 1.25
    out = pa.rotary_append(b.q, b.k, b.v, kc, vc, b.tables.cuda(), i32(b.ctx), i32(b.qs), freqs,
                           interleaved=pairs, amplitude=amp)
    assert pa.get_device_error() == 0
    close(out[:b.n].cpu(), *turned64(b.q[:b.n].cpu(), b.pos, f, pairs, amp), b.dt)
    blk, row = b.slots()
    close(kc.cpu()[blk, :, row], *turned64(b.k[:b.n].cpu(), b.pos, f, pairs, amp), b.dt)
    assert torch.equal(vc.cpu()[blk, :, row], b.v[:b.n].cpu())
    for new, old in ((kc, b.kc), (vc, b.vc)):  # nothing else has changed
        new, old = new.cpu(), old.cpu()
        new[blk, :, row] = old[blk, :, row]
        assert torch.equal(new, old)
    # without the cache write: the same bits
    o2, k2 = pa.rotary(b.q, b.k, i32(b.ctx), i32(b.qs), freqs, interleaved=pairs, amplitude=amp)
    assert torch.equal(o2[:b.n], out[:b.n]) and torch.equal(k2[:b.n].cpu(), kc.cpu()[blk, :, row])
    # the values behind rotary_dim as they were
    assert torch.equal(out[:b.n, :, rd:], b.q[:b.n, :, rd:])


@pytest.mark.parametrize("pairs", [False, True])
def test_in_place_and_rows_behind_the_last(pairs):
    b = Batch([3, 1, 9], [5, 0, 70], 4, 2, 64, 16, "bf16", True, extra=6)
    freqs, _ = pa.rotary_frequencies(64)
    want, kwant = pa.rotary(b.q, b.k, i32(b.ctx), i32(b.qs), freqs, interleaved=pairs)
    before = [t.clone() for t in (b.q, b.k, b.v)]
    out, key = pa.rotary(b.q, b.k, i32(b.ctx), i32(b.qs), freqs, interleaved=pairs, out=b.q, key_out=b.k)
    assert out.data_ptr() == b.q.data_ptr()
    assert torch.equal(b.q[:b.n], want[:b.n]) and torch.equal(b.k[:b.n], kwant[:b.n])
    for t, old in zip((b.q, b.k), before):
        assert torch.equal(t[b.n:], old[b.n:])
    assert torch.equal(b.v, before[2])
    q = before[0].contiguous()
    pa.rotary_append(q, before[1], before[2], b.kc, b.vc, b.tables.cuda(), i32(b.ctx), i32(b.qs), freqs,
                     interleaved=pairs, out=q)
    assert torch.equal(q[:b.n], want[:b.n]) and torch.equal(q[b.n:], before[0][b.n:])


def test_negative_zero_infinite_and_nan_values_stay_where_they_are():
    b = Batch([4], [0], 1, 1, 64, 16, "fp16", False)
    b.q[1, 0, 3], b.q[2, 0, 40], b.k[3, 0, 63] = math.nan, math.inf, -math.inf
    freqs, _ = pa.rotary_frequencies(32)
    out, key = pa.rotary(b.q, b.k, i32(b.ctx), i32(b.qs), freqs)
    assert out[1, 0].isnan().nonzero().flatten().tolist() == [3, 19]  # its pair alone
    assert out[2, 0, 40] == math.inf and key[3, 0, 63] == -math.inf
    assert out[0, 0].isfinite().all() and torch.equal(out[0], b.q[0])  # position 0: not turned


@pytest.mark.parametrize("kind,more", [
    ("linear", dict()), ("bands", dict(low=1.0, high=4.0, trained=8192)),
    ("ramp", dict(slow=1.0, fast=32.0, trained=4096)), ("ramp", dict(slow=1.0, fast=32.0, trained=4096, amplitude=1.0))])
def test_stretched_contexts(kind, more):
    rd, base, factor = 64, 10000.0, 8.0
    freqs, amp = pa.rotary_frequencies(rd, base, dict(kind=kind, factor=factor, **more))
    f = angles64(rd, base)
    for i in range(rd // 2):  # the definition, pair by pair
        x = float(f[i])
        if kind == "linear":
            f[i] = x / factor
        elif kind == "bands":
            turns = 8192 * x / (2 * math.pi)
            a = 0.0 if turns < 1 else (1.0 if turns > 4 else (turns - 1) / 3)
            f[i] = (1 - a) * x / factor + a * x
        else:
            lo = math.floor(rd * math.log(4096 / (32 * 2 * math.pi)) / (2 * math.log(base)))
            hi = math.ceil(rd * math.log(4096 / (1 * 2 * math.pi)) / (2 * math.log(base)))
            a = 0.0 if i <= lo else (1.0 if i >= hi else (i - lo) / (hi - lo))
            f[i] = a * x / factor + (1 - a) * x
    want = 0.1 * math.log(factor) + 1 if kind == "ramp" and "amplitude" not in more else 1.0
    assert abs(amp - want) < 1e-12
    b = Batch([5, 2], [20000, 60000], 2, 1, 64, 16, "bf16", True)
    out, _ = pa.rotary(b.q, b.k, i32(b.ctx), i32(b.qs), freqs, amplitude=amp)
    close(out[:b.n].cpu(), *turned64(b.q[:b.n].cpu(), b.pos, f, False, amp), b.dt)


def test_impossible_sequences_are_skipped_and_told():
    b = Batch([2, 2, 2, 2], [5, 5, 5, 5], 2, 1, 64, 16, "bf16", False, extra=0)
    freqs, _ = pa.rotary_frequencies(64)
    cap = b.tables.shape[1] * 16

    def call(ctx, qs, tables=b.tables):
        kc, vc = b.kc.clone(), b.vc.clone()
        out = torch.full_like(b.q, 7.0)
        pa.get_device_error()
        pa.rotary_append(b.q, b.k, b.v, kc, vc, tables.cuda(), i32(ctx), i32(qs), freqs, out=out)
        changed = [s for s in range(4) if int(b.tables[s, 0]) in
                   ((kc != b.kc) | (vc != b.vc)).flatten(1).any(1).nonzero().flatten().tolist()]
        return out, changed, pa.get_device_error()

    good = [7, 7, 7, 7]
    for ctx in ([7, 1, 7, 7], [7, -4, 7, 7], [7, cap + 1, 7, 7]):
        out, changed, err = call(ctx, b.qs)
        assert err == pa.DEVERR_BAD_CONTEXT and changed == [0, 2, 3]
        assert (out[2:4] == 7.0).all() and (out[[0, 1, 4, 5, 6, 7]] != 7.0).any()
    out, changed, err = call(good, [0, 2, 4, 6, 9])
    assert err == pa.DEVERR_BAD_CONTEXT and changed == [0, 1, 2] and (out[6:] == 7.0).all()
    out, changed, err = call(good, [0, 2, 1, 6, 8])
    assert err == pa.DEVERR_BAD_CONTEXT and 1 not in changed
    t = b.tables.clone()
    t[2, 0] = 1000
    out, changed, err = call(good, b.qs, t)
    assert err == pa.DEVERR_BAD_BLOCK and changed == [0, 1, 3]
    assert torch.equal(out, call(good, b.qs)[0])  # q is turned all the same


def test_many_sequences():
    rows = [1 if s % 3 else 0 for s in range(1000)]
    b = Batch(rows, [(7 * s) % 300 for s in range(1000)], 2, 1, 64, 16, "bf16", False)
    freqs, _ = pa.rotary_frequencies(64)
    out, _ = pa.rotary(b.q, b.k, i32(b.ctx), i32(b.qs), freqs)
    close(out[:b.n].cpu(), *turned64(b.q[:b.n].cpu(), b.pos, angles64(64, 10000.0), False, 1.0), b.dt)


def test_other_stream_plan_and_graph():
    b = Batch([2, 1], [30, 0], 4, 2, 128, 16, "bf16", True)
    freqs, _ = pa.rotary_frequencies(128)
    ctx, qs, t = i32(b.ctx), i32(b.qs), b.tables.cuda()
    want = pa.rotary_append(b.q, b.k, b.v, b.kc, b.vc, t, ctx, qs, freqs)
    kwant = b.kc.clone()
    b.kc.zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = pa.rotary_append(b.q, b.k, b.v, b.kc, b.vc, t, ctx, qs, freqs, stream=side)
    side.synchronize()
    blk, row = b.slots()
    assert torch.equal(out[:b.n], want[:b.n])
    assert torch.equal(b.kc.cpu()[blk, :, row], kwant.cpu()[blk, :, row])
    plan = pa.rotary_append(b.q, b.k, b.v, b.kc, b.vc, t, ctx, qs, freqs, out=torch.zeros_like(out), plan=True)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.run(torch.cuda.current_stream())
    b.q.copy_(b.q.flip(2))
    g.replay()
    assert torch.equal(plan.out[:b.n], pa.rotary(b.q, b.k, ctx, qs, freqs)[0][:b.n])


def test_refusals():
    b = Batch([2], [0], 2, 1, 64, 16, "bf16", False, extra=0)
    freqs, _ = pa.rotary_frequencies(64)
    ctx, qs, t = i32(b.ctx), i32(b.qs), b.tables.cuda()

    def call(q=b.q, k=b.k, v=b.v, f=freqs, **kw):
        return pa.rotary_append(q, k, v, b.kc, b.vc, t, ctx, qs, f, **kw)
    with pytest.raises(pa.PagedAttentionError):
        call(f=freqs[:12])  # 24 of 64 values: not a multiple of 16
    with pytest.raises(pa.PagedAttentionError):
        call(f=pa.rotary_frequencies(128)[0])
    with pytest.raises(pa.PagedAttentionError):
        call(amplitude=math.nan)
    with pytest.raises(ValueError):
        call(q=b.q.half())
    with pytest.raises(ValueError):
        call(k=b.k[:1])
    with pytest.raises(ValueError):
        call(q=b.q.cpu())
    with pytest.raises(ValueError):
        call(f=freqs.int())
    with pytest.raises(ValueError):  # heads not contiguous
        call(q=torch.empty(2, 64, 2, dtype=torch.bfloat16, device="cuda").transpose(1, 2))
    odd = torch.empty(2, 2 * 64 + 4, dtype=torch.bfloat16, device="cuda")[:, :128].unflatten(1, (2, 64))
    with pytest.raises(pa.PagedAttentionError):  # rows 132 values apart
        call(q=odd)
    off = torch.empty(2 * 128 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(2, 2, 64)
    with pytest.raises(pa.PagedAttentionError):  # not 16-byte aligned
        call(q=off)
    none = b.q[:0]
    assert pa.rotary(none, b.k[:0], ctx, qs, freqs)[0].shape == (0, 2, 64)


def test_rows_that_belong_to_no_sequence():
    b = Batch([3, 1], [5, 0], 4, 2, 64, 16, "bf16", True, extra=6)
    freqs, _ = pa.rotary_frequencies(64)
    q0 = b.q.clone()
    pa.get_device_error()
    pa.rotary(b.q, b.k, i32([8, 1]), i32([2, 5, 6]), freqs, out=b.q, key_out=b.k)
    assert pa.get_device_error() == 0
    assert torch.equal(b.q[[0, 1, 6, 7, 8, 9]], q0[[0, 1, 6, 7, 8, 9]])
    pos = torch.tensor([5, 6, 7, 0])
    close(b.q[2:6].cpu(), *turned64(q0[2:6].cpu(), pos, angles64(64, 10000.0), False, 1.0), b.dt)
    q1 = b.q.clone()
    pa.rotary(b.q, b.k, i32([8, 1]), i32([0, 0, 0]), freqs, out=b.q, key_out=b.k)
    assert torch.equal(b.q, q1)


def test_two_streams_at_once():
    batches = [Batch([40, 1, 7], [5, 100, 0], 8, 2, 128, 16, "bf16", True, seed=s) for s in (1, 2)]
    freqs, _ = pa.rotary_frequencies(128)
    args = [(b.q, b.k, b.v, b.kc, b.vc, b.tables.cuda(), i32(b.ctx), i32(b.qs), freqs) for b in batches]
    want = [pa.rotary_append(*a).clone() for a in args]
    caches = [b.kc.clone() for b in batches]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [(i, pa.rotary_append(*args[i], stream=streams[i])) for _ in range(20) for i in (0, 1)]
    torch.cuda.synchronize()
    assert all(torch.equal(o[:batches[i].n], want[i][:batches[i].n]) for i, o in got)
    assert all(torch.equal(b.kc, c) for b, c in zip(batches, caches))


@pytest.mark.parametrize("qs, written", [
    ([0, 8, 2, 4, 6], [0, 1, 2, 3, 4, 5, 6, 7]),  # sequence 1 decreases: every row is sequence 0's
    ([0, 30, 2, 4, 6], [2, 3, 4, 5]),              # rows 6 and 7 are behind every span
    ([0, -3, 2, 4, 6], [2, 3, 4, 5]),
    ([6, 8, 1, 3, 3], [1, 2, 6, 7]),
])
def test_rows_beside_impossible_spans(qs, written):
    # contexts that fill the tables: a row taken for a place behind its sequence's last would be past them
    b = Batch([2, 2, 2, 2], [5, 5, 5, 5], 2, 1, 64, 16, "bf16", False, extra=0)
    freqs, _ = pa.rotary_frequencies(64)
    tables = torch.arange(4, dtype=torch.int32).reshape(4, 1)
    kc, vc = (torch.zeros(4, 1, 16, 64, dtype=b.dt, device="cuda") for _ in range(2))
    out = torch.full_like(b.q, 7.0)
    pa.get_device_error()
    pa.rotary_append(b.q, b.k, b.v, kc, vc, tables.cuda(), i32([16] * 4), i32(qs), freqs, out=out)
    assert pa.get_device_error() == pa.DEVERR_BAD_CONTEXT
    assert (out != 7.0).flatten(1).any(1).nonzero().flatten().tolist() == written
    # each row in the slot of the sequence that holds it, and no other slot
    slots = {}
    for r in written:
        s = next(s for s in range(4) if 0 <= qs[s] <= r < qs[s + 1] <= 8)
        slots[(s, 16 - qs[s + 1] + r)] = r
    want = torch.zeros_like(vc)
    for (s, row), r in slots.items():
        want[s, 0, row] = b.v[r, 0]
    assert torch.equal(vc, want)
    other = torch.full_like(b.q, 7.0)
    pa.rotary(b.q, b.k, i32([16] * 4), i32(qs), freqs, out=other, key_out=torch.empty_like(b.k))
    assert pa.get_device_error() == pa.DEVERR_BAD_CONTEXT and torch.equal(other, out)
