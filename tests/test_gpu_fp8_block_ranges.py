"""FP8 blocks with block scales at the ends of their ranges: many short prompts, more sequences
than lanes, spans that the call bounds, scales far apart, one long sequence cut into many pieces,
not-a-number codes, caches past 4 GiB, captured and replayed steps, and calls on two streams at
once."""
import numpy as np
import pytest
import torch

import paged_kv_cache_149_gb300 as pa
from fp8_block_harness import DTYPE, Batch, bound, dev, dev16, rows16, values
from gpu_harness import device_error
from oracle import fp8_block as fb
from oracle.formats import decode_bits

pytestmark = pytest.mark.gpu

P_STEP = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _lib(libpa):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    device_error()


def upload(caches):
    return [dev(x) for x in caches]


def check_rows(b, caches, got, q, qs, scale, rows_of):
    """got [rows, Hq, d] float64 against each asked row's own sum over the cache."""
    for s, c in enumerate(int(x) for x in b.ctx):
        k = fb.logical_rows(caches[0], caches[2], b.tables[s], c)
        v = fb.logical_rows(caches[1], caches[3], b.tables[s], c)
        new = int(qs[s + 1] - qs[s])
        for i in sorted(set(rows_of(new)) & set(range(new))):
            n = c - (new - 1 - i)
            row = int(qs[s]) + i
            want = fb.attend(q[row], k[:n], v[:n], scale)
            off = np.abs(got[row] - want)
            most = bound(q[row], k[:n], v[:n], scale, want, b.dtype, P_STEP[b.dtype])
            assert (off <= most).all(), (s, c, i, float((off / most).max()))


def prefill(b, caches, new, spread=0, most=None):
    qs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q_bits = rows16(b.rng, (int(qs[-1]), b.hq, b.d), b.dtype, spread)
    out = torch.full((len(q_bits), b.hq, b.d), 7.0, dtype=DTYPE[b.dtype], device="cuda")
    pa.prefill_fp8_block(dev16(q_bits, b.dtype), *upload(caches), dev(b.tables), dev(b.ctx), dev(qs),
                         1.0 / np.sqrt(b.d), int(max(new)) if most is None else most, out=out)
    return values(out, b.dtype), decode_bits(q_bits, b.dtype), qs


# --------------------------------------------------------------------------------- prefill

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_many_short_prompts(dtype):
    """Items of one to three key tiles follow one another on an SM; each row of q has a power of
    two of its own, so that a row's factor taken from another item would show."""
    n = 300
    ctx = [1 + (37 * i) % 64 if i % 3 else 1 + (53 * i) % 180 for i in range(n)]
    b = Batch(ctx, 8, 4, 128, 16, dtype, seed=1)
    caches = b.written()
    got, q, qs = prefill(b, caches, ctx, spread=3)
    assert device_error() == 0
    check_rows(b, caches, got, q, qs, 1.0 / np.sqrt(128), lambda new: (0, new // 2, new - 1))


def test_more_sequences_than_lanes_keep_apart():
    ctx = [1 + i % 5 for i in range(1200)]
    new = [1 if i % 7 else min(3, c) for i, c in enumerate(ctx)]
    new[40] = new[900] = 0
    b = Batch(ctx, 2, 1, 64, 8, "fp16", seed=2)
    caches = b.written()
    got, q, qs = prefill(b, caches, new)
    assert device_error() == 0
    check_rows(b, caches, got, q, qs, 0.125, lambda n: range(n))


@pytest.mark.parametrize("hq,hkv", [(64, 1), (33, 1), (96, 2), (65, 5)])
@pytest.mark.parametrize("d", [64, 128])
def test_prefill_of_wide_and_odd_groups(hq, hkv, d):
    b = Batch([70, 9, 200], hq, hkv, d, 16, "bf16", seed=hq)
    caches = b.written()
    got, q, qs = prefill(b, caches, [70, 4, 30])
    assert device_error() == 0
    check_rows(b, caches, got, q, qs, 1.0 / np.sqrt(d), lambda n: (0, n // 2, n - 1))


def test_spans_past_max_query_len_and_past_the_rows():
    """Rows past max_query_len's query blocks are not computed; a span that is not the call's
    touches nothing and is reported."""
    b = Batch([300, 40], 4, 1, 128, 16, "fp16", seed=3)
    caches = b.written()
    got, q, qs = prefill(b, caches, [300, 40], most=32)  # one query block of each
    assert device_error() == 0
    k = fb.logical_rows(caches[0], caches[2], b.tables[0], 300)
    v = fb.logical_rows(caches[1], caches[3], b.tables[0], 300)
    for i in (0, 31):
        want = fb.attend(q[i], k[:i + 1], v[:i + 1], 1.0 / np.sqrt(128))
        assert (np.abs(got[i] - want) <= bound(q[i], k[:i + 1], v[:i + 1], 1.0 / np.sqrt(128), want, "fp16")).all()
    assert (got[64:300] == 7).all()
    qs = np.array([0, 300, 500], np.int32)  # the second span ends past the 340 rows of q
    out = torch.full((340, 4, 128), 7.0, dtype=torch.float16, device="cuda")
    q16 = torch.randn(340, 4, 128, device="cuda").half()
    pa.prefill_fp8_block(q16, *upload(caches), dev(b.tables), dev(b.ctx), dev(qs), 0.1, 300, out=out)
    assert device_error() == pa.DEVERR_BAD_CONTEXT
    assert (out[300:] == 7).all() and (out[:300] != 7).any()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_prefill_over_scales_far_apart_and_odd(dtype):
    """V scales that grow by 2^9 and more from tile to tile (the sums' reference moves), shrink
    again, and scales that are no powers of two."""
    b = Batch([700, 450], 4, 2, 128, 16, dtype, seed=4)
    k8, v8, ks, vs = b.written()
    for s in range(2):
        for j in range(-(-int(b.ctx[s]) // 16)):
            blk = b.tables[s, j]
            vs[blk] = [2.0 ** (3 * (j // 4) - 20), 2.0 ** (-5 * (j % 7)) * 1.37]
            ks[blk] *= np.float32(1.19) if j % 2 else np.float32(0.83)
    caches = (k8, v8, ks, vs)
    got, q, qs = prefill(b, caches, [700, 120])
    assert device_error() == 0
    check_rows(b, caches, got, q, qs, 1.0 / np.sqrt(128), lambda n: (0, 5, n // 2, n - 1))


# --------------------------------------------------------------------------------- decode

@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (16, 1, 128), (14, 2, 64), (8, 4, 128), (32, 1, 64)])
@pytest.mark.parametrize("ctx", [[9000], [5000, 1, 333]])
def test_decode_of_few_long_sequences(hq, hkv, d, ctx):
    b = Batch(ctx, hq, hkv, d, 16, "fp16", seed=hq)
    caches = b.written()
    q_bits = rows16(b.rng, (len(ctx), hq, d), "fp16")
    q, scale = decode_bits(q_bits, "fp16"), 1.0 / np.sqrt(d)
    got = values(pa.decode_fp8_block(dev16(q_bits, "fp16"), *upload(caches), dev(b.tables), dev(b.ctx), scale), "fp16")
    assert device_error() == 0
    check_rows(b, caches, got, q, np.arange(len(ctx) + 1), scale, lambda n: range(n))


@pytest.mark.parametrize("hq,hkv,d", [(7, 1, 64), (48, 3, 128), (10, 5, 64), (12, 12, 128), (4, 2, 128)])
@pytest.mark.parametrize("n", [3, 40, 330])
def test_decode_of_short_sequences_with_few_or_odd_heads(hq, hkv, d, n):
    """Sequences that one warp takes among others that several share, contexts that are invalid
    and a block outside the pool among them."""
    ctx = [1 + (29 * i) % 70 if i % 5 else 1 + (311 * i) % 900 for i in range(n)]
    b = Batch(ctx, hq, hkv, d, 8, "bf16", seed=n)
    caches = b.written()
    q_bits = rows16(b.rng, (n, hq, d), "bf16")
    q, scale = decode_bits(q_bits, "bf16"), 1.0 / np.sqrt(d)
    tables, lens = b.tables.copy(), b.ctx.copy()
    zeros = [1] if n == 3 else [1, 7, n // 2, n - 1]
    lens[zeros[0]] = 0
    for s in zeros[1:]:
        tables[s, (lens[s] - 1) // 8] = -1 if s % 2 else b.nb
    out = pa.decode_fp8_block(dev16(q_bits, "bf16"), *upload(caches), dev(tables), dev(lens), scale)
    got = values(out, "bf16")
    assert device_error() == pa.DEVERR_BAD_CONTEXT | (pa.DEVERR_BAD_BLOCK if n > 3 else 0)
    assert (got[zeros] == 0).all()
    keep = np.setdiff1d(np.arange(n), zeros)
    b.ctx, b.tables = b.ctx[keep], b.tables[keep]
    check_rows(b, caches, got[keep], q[keep], np.arange(len(keep) + 1), scale, lambda m: range(m))


@pytest.mark.parametrize("hq,hkv", [(8, 2), (8, 8), (4, 1)])
@pytest.mark.parametrize("ctx", [40, 4000])
def test_a_nan_code_reaches_its_head_and_no_other(hq, hkv, ctx):
    """Whole and cut between SMs: NaN in a key makes its head's queries NaN, NaN in a value its
    column; behind the context it is not read."""
    b = Batch([ctx], hq, hkv, 64, 16, "fp16", seed=5)
    k8, v8, ks, vs = b.written()
    q = dev16(rows16(b.rng, (1, hq, 64), "fp16"), "fp16")
    run = lambda k, v: pa.decode_fp8_block(q, dev(k), dev(v), dev(ks), dev(vs), dev(b.tables), dev(b.ctx), 0.125)  # noqa: E731
    plain = run(k8, v8)
    assert torch.isfinite(plain).all()
    t, G = ctx // 2, hq // hkv
    kn, vn = k8.copy(), v8.copy()
    kn[b.tables[0, t // 16], 0, t % 16, 9] = 0x7F
    vn[b.tables[0, t // 16], 0, t % 16, 9] = 0xFF
    out = run(kn, v8)
    assert torch.isnan(out[:, :G]).all() and torch.equal(out[:, G:], plain[:, G:])
    out = run(k8, vn)
    assert torch.isnan(out[:, :G, 9]).all() and torch.equal(out[:, G:], plain[:, G:])
    out[:, :G, 9] = plain[:, :G, 9]
    assert torch.equal(out, plain) and device_error() == 0


def test_a_nan_key_behind_a_token_does_not_reach_it():
    b = Batch([100], 4, 2, 128, 16, "bf16", seed=6)
    k8, v8, ks, vs = b.written()
    q = dev16(rows16(b.rng, (100, 4, 128), "bf16"), "bf16")
    qs = dev([0, 100], np.int32)
    run = lambda k: pa.prefill_fp8_block(q, dev(k), dev(v8), dev(ks), dev(vs), dev(b.tables), dev(b.ctx), qs, 0.1, 100)  # noqa: E731
    plain = run(k8)
    kn = k8.copy()
    kn[b.tables[0, 70 // 16], 1, 70 % 16, 3] = 0x7F
    out = run(kn)
    assert torch.isnan(out[70:, 2:]).all()
    assert torch.equal(out[:70], plain[:70]) and torch.equal(out[:, :2], plain[:, :2])
    assert device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 128), (7, 1, 64), (2, 2, 128)])
@pytest.mark.parametrize("ctx,new,at", [(100, 100, (70,)), (500, 300, (10, 199, 200, 350, 499)), (700, 1, (699, 3)),
                                        (64, 2, (62, 63)), (900, 900, (0, 63, 64, 640))])
def test_a_nan_value_reaches_the_tokens_behind_it_only(dtype, hq, hkv, d, ctx, new, at):
    """NaN in a value's column: NaN in that column for its head's queries from its token on, and
    every other output as it is with a zero there."""
    b = Batch([ctx, 40], hq, hkv, d, 16, dtype, seed=7)
    k8, v8, ks, vs = b.written()
    qs = np.array([0, new, new + 40], np.int32)
    q = dev16(rows16(b.rng, (new + 40, hq, d), dtype), dtype)
    run = lambda v: pa.prefill_fp8_block(q, dev(k8), dev(v), dev(ks), dev(vs), dev(b.tables), dev(b.ctx), dev(qs), 0.1, max(new, 40))  # noqa: E731
    vz, vn, G = v8.copy(), v8.copy(), hq // hkv
    nan = np.zeros((new + 40, hq, d), bool)
    for i, t in enumerate(at):
        h, c = i % hkv, (5 + 13 * i) % d
        vz[b.tables[0, t // 16], h, t % 16, c] = 0
        vn[b.tables[0, t // 16], h, t % 16, c] = 0x7F if i % 2 else 0xFF
        nan[max(0, t - (ctx - new)):new, h * G:(h + 1) * G, c] = True
    want, got = run(vz), run(vn)
    nan = torch.from_numpy(nan).cuda()
    assert torch.isnan(got[nan]).all() and torch.equal(got[~nan], want[~nan])
    assert torch.isfinite(want).all() and device_error() == 0


# --------------------------------------------------------------------------------- large caches

def test_caches_past_4_gib():
    """The same step over the first blocks of a small pool and the last of one whose caches hold
    more than 2^32 codes each: the same tables apart from the block ids, codes, scales, outputs."""
    hkv, B, d, dt = 2, 16, 128, torch.bfloat16
    big, n = (1 << 32) // (hkv * B * d) + 200, 64
    gen = torch.Generator(device="cuda").manual_seed(7)
    lens, news = dev([500, 260, 3], np.int32), dev([500, 30, 3], np.int32)
    past = 230
    rows = lambda h: torch.randn(533, h, d, generator=gen, device="cuda").to(dt)  # noqa: E731
    key, value, q = rows(hkv), rows(hkv), rows(4)
    old = torch.randn(past, hkv, d, generator=gen, device="cuda").to(dt)
    res = []
    for nb in (n, big):
        ids = torch.arange(nb - 1, nb - 1 - n, -1, dtype=torch.int32, device="cuda")
        k8, v8 = (torch.zeros(nb, hkv, B, d, dtype=torch.uint8, device="cuda") for _ in range(2))
        ks, vs = (torch.empty(nb, hkv, device="cuda") for _ in range(2))
        tables = torch.full((3, 40), -1, dtype=torch.int32, device="cuda")
        slots = torch.empty(600, dtype=torch.int64, device="cuda")
        before, _ = pa.build_step(dev([0, past, 0], np.int32), dev([0, past, 0], np.int32), ids,
                                  dev([0], np.int32), tables, B, nb, slots)
        pa.append_fp8_block(old, old, k8, v8, ks, vs, tables, dev([0, past, 0], np.int32), before)
        qs, left = pa.build_step(news, lens, ids, dev([-(-past // B)], np.int32), tables, B, nb, slots)
        pa.append_fp8_block(key, value, k8, v8, ks, vs, tables, lens, qs)
        o1 = pa.prefill_fp8_block(q, k8, v8, ks, vs, tables, lens, qs, 0.09, 500)
        o2 = pa.decode_fp8_block(q[:3], k8, v8, ks, vs, tables, lens, 0.09)
        used = int(left)
        pair = torch.stack([ids[:1], ids[n - 1:n]], 1).contiguous()
        pa.copy_blocks_fp8_block(k8, v8, ks, vs, pair)
        assert torch.equal(k8[int(ids[n - 1])], k8[int(ids[0])]) and torch.equal(vs[int(ids[n - 1])], vs[int(ids[0])])
        at = ids[:used].long()
        res.append((o1, o2, (slots - (nb - n) * B)[:533], torch.where(tables >= 0, tables - (nb - n), tables),
                    k8[at], v8[at], ks[at], vs[at]))
        assert device_error() == 0
    torch.cuda.synchronize()
    for a, c in zip(*res):
        assert torch.equal(a, c)


# --------------------------------------------------------------------------------- graphs, streams

def _step(b, hq, T):
    """The tensors of one serving step over an empty pool."""
    n = len(b.ctx)
    st = dict(caches=upload(b.empty()), tables=torch.full((n, T), -1, dtype=torch.int32, device="cuda"),
              free=dev(np.arange(b.nb, dtype=np.int32)), start=dev([0], np.int32),
              slots=torch.empty(int(b.qs[-1]) + 5, dtype=torch.int64, device="cuda"),
              key=dev16(b.key, b.dtype), value=dev16(b.value, b.dtype),
              q=dev16(rows16(b.rng, (int(b.qs[-1]), hq, b.d), b.dtype), b.dtype), lens=dev(b.ctx))
    st["qs"], st["left"] = torch.zeros(n + 1, dtype=torch.int32, device="cuda"), dev([0], np.int32)
    st["out"] = torch.zeros_like(st["q"])
    st["one"] = torch.zeros_like(st["q"][:n])
    st["ws"] = pa.make_workspace(hq, b.hkv, b.d)
    return st


def _run(st, B, nb, most, stream=None):
    pa.build_step(st["lens"], st["lens"], st["free"], st["start"], st["tables"], B, nb, st["slots"],
                  query_start=st["qs"], free_next=st["left"], stream=stream)
    pa.append_fp8_block(st["key"], st["value"], *st["caches"], st["tables"], st["lens"], st["qs"], stream=stream)
    pa.prefill_fp8_block(st["q"], *st["caches"], st["tables"], st["lens"], st["qs"], 0.1, most, out=st["out"], stream=stream)
    pa.decode_fp8_block(st["q"][:len(st["lens"])], *st["caches"], st["tables"], st["lens"], 0.1, out=st["one"],
                        workspace=st["ws"], stream=stream)
    pa.copy_blocks_fp8_block(*st["caches"], st["pair"], stream=stream)


RESULT = ("tables", "slots", "qs", "left", "out", "one")


def _results(st, used):
    return [st[k].clone() for k in RESULT] + [t[used].clone() for t in st["caches"]]


def test_a_captured_step_replayed_over_other_lengths():
    b = Batch([130, 64, 7, 300], 8, 2, 128, 16, "bf16", seed=8)
    b.nb += 10
    st = _step(b, 8, 24)
    st["pair"] = dev([[0, b.nb - 1]], np.int32)
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    _run(st, 16, b.nb, 300)
    torch.cuda.synchronize()
    with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
        _run(st, 16, b.nb, 300, stream=side)
    for lens in ([130, 64, 7, 300], [1, 0, 300, 200], [16, 17, 0, 0]):
        got = []
        for run in (g.replay, lambda: _run(st, 16, b.nb, 300)):
            st["lens"].copy_(dev(lens, np.int32))
            st["tables"].fill_(-1)
            st["out"].fill_(3)
            for c in st["caches"]:
                c.view(torch.uint8).fill_(0x7F)
            run()
            torch.cuda.synchronize()
            used = torch.arange(int(st["left"]), device="cuda")
            got.append(_results(st, torch.cat([used, used.new_tensor([b.nb - 1])])))
        assert device_error() == (pa.DEVERR_BAD_CONTEXT if 0 in lens else 0)  # (decode of no tokens)
        for a, c in zip(*got):
            assert torch.equal(a, c) or torch.equal(a.float().nan_to_num(5), c.float().nan_to_num(5))
        assert (st["out"][sum(lens):] == 3).all()


def test_steps_on_two_streams_at_once():
    """Two steps with tensors and workspaces of their own, many times over on two streams, give
    what each gives alone."""
    sts, alone, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    shapes = [([900, 64, 300, 1], 8, 2, 128, 16, "bf16"), ([33, 1500, 2], 4, 4, 64, 8, "fp16")]
    for i, (ctx, hq, hkv, d, B, dtype) in enumerate(shapes):
        b = Batch(ctx, hq, hkv, d, B, dtype, seed=20 + i)
        st = _step(b, hq, -(-max(ctx) // B))
        st.update(pair=dev([[0, b.nb - 1]], np.int32), B=B, nb=b.nb, most=max(ctx))
        _run(st, B, b.nb, st["most"])
        torch.cuda.synchronize()
        st["used"] = torch.cat([torch.arange(int(st["left"])), torch.tensor([b.nb - 1])]).cuda()
        alone.append(_results(st, st["used"]))
        sts.append(st)
    for _ in range(20):
        for st, stream in zip(sts, streams):
            with torch.cuda.stream(stream):
                st["tables"].fill_(-1)
                _run(st, st["B"], st["nb"], st["most"])
    torch.cuda.synchronize()
    assert device_error() == 0
    for st, want in zip(sts, alone):
        for a, c in zip(_results(st, st["used"]), want):
            assert torch.equal(a, c)


def test_outputs_are_allocated_for_the_stream_of_the_call():
    """The memory of a tensor freed on the current stream, with work on it still under way there,
    is not handed to a call on another stream."""
    b = Batch([130, 64, 7, 300], 8, 2, 128, 16, "bf16", seed=10)
    st = _step(b, 8, 24)
    st["pair"] = dev([[0, b.nb - 1]], np.int32)
    _run(st, 16, b.nb, 300)
    torch.cuda.synchronize()
    side, args = torch.cuda.Stream(), (*st["caches"], st["tables"], st["lens"])
    for _ in range(10):
        junk = torch.empty_like(st["out"])
        for _ in range(50):
            junk.fill_(9)
        del junk
        out = pa.prefill_fp8_block(st["q"], *args, st["qs"], 0.1, 300, stream=side)
        one = pa.decode_fp8_block(st["q"][:4], *args, 0.1, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, st["out"]) and torch.equal(one, st["one"])
    assert device_error() == 0


def test_planned_calls_run_again_on_any_stream():
    b = Batch([130, 64, 7, 300], 8, 2, 128, 16, "fp16", seed=9)
    st = _step(b, 8, 24)
    st["pair"] = dev([[0, b.nb - 1]], np.int32)
    _run(st, 16, b.nb, 300)
    torch.cuda.synchronize()
    used = torch.arange(int(st["left"]), device="cuda")
    want = _results(st, used)
    plans = [
        pa.build_step(st["lens"], st["lens"], st["free"], st["start"], st["tables"], 16, b.nb, st["slots"],
                      query_start=st["qs"], free_next=st["left"], plan=True),
        pa.append_fp8_block(st["key"], st["value"], *st["caches"], st["tables"], st["lens"], st["qs"], plan=True),
        pa.prefill_fp8_block(st["q"], *st["caches"], st["tables"], st["lens"], st["qs"], 0.1, 300, out=st["out"], plan=True),
        pa.decode_fp8_block(st["q"][:4], *st["caches"], st["tables"], st["lens"], 0.1, out=st["one"], plan=True)]
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream()):
        st["tables"].fill_(-1)
        for k in ("out", "one", "slots", "qs"):
            st[k].zero_()
        torch.cuda.synchronize()
        for p in plans:
            p.run(stream)
        torch.cuda.synchronize()
        for a, c in zip(_results(st, used), want):
            assert torch.equal(a, c)
    assert device_error() == 0
