"""Host side of the drafted step: refusals before any CUDA call, angles as exact fractions of a
turn, and the pool's truncation."""
import math
import random
from fractions import Fraction

import numpy as np
import pytest

# 2 pi, to 60 digits
TWO_PI = 2 * Fraction("3.141592653589793238462643383279502884197169399375105820974944")


def test_frequencies_are_rounded_once(libpa):
    rng = random.Random(1)
    f = [rng.random() * 10.0 ** rng.uniform(-12, 0) for _ in range(500)]
    f += [0.0, 1.0, -1.0, -0.37, 1e6, 2 * math.pi, 1e-300, 5e-324, 500000.0 ** -0.5]
    src, out = np.array(f), np.zeros(len(f), np.uint64)
    assert libpa.lib().pa_rotary_frequencies(src.ctypes.data, len(f), out.ctypes.data) == 0
    for x, got in zip(f, out.tolist()):
        d = (Fraction(got) - Fraction(x) / TWO_PI * 2 ** 64) % 2 ** 64
        d = min(d, 2 ** 64 - d)
        assert d <= Fraction(1, 2) + Fraction(1, 1000)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, 1.1e6])
def test_frequencies_refused(libpa, bad):
    src, out = np.array([0.5, bad]), np.zeros(2, np.uint64)
    assert libpa.lib().pa_rotary_frequencies(src.ctypes.data, 2, out.ctypes.data) == libpa.PA_ERR_ARG
    assert (out == 0).all()
    assert libpa.lib().pa_rotary_frequencies(None, 1, out.ctypes.data) == libpa.PA_ERR_ARG
    assert libpa.lib().pa_rotary_frequencies(None, 0, None) == 0


def test_frequencies_of_a_model(libpa):
    freqs, amp = libpa.rotary_frequencies(64, 10000.0, device="cpu")
    assert amp == 1.0 and freqs.shape == (32,)
    assert freqs[0] == round(2 ** 64 / (2 * math.pi) / 2 ** 11) * 2 ** 11 or abs(
        int(freqs[0]) - float(2 ** 64 / TWO_PI)) < 2 ** 12
    for bad in (dict(rotary_dim=63), dict(rotary_dim=0), dict(rotary_dim=64, base=1.0),
                dict(rotary_dim=64, scaling=dict(kind="linear", factor=0.0)),
                dict(rotary_dim=64, scaling=dict(kind="linear", factor=2.0, more=1)),
                dict(rotary_dim=64, scaling=dict(kind="other", factor=2.0)),
                dict(rotary_dim=64, scaling=dict(kind="bands", factor=2.0, low=4.0, high=1.0, trained=100))):
        with pytest.raises(ValueError):
            libpa.rotary_frequencies(device="cpu", **bad)


# (addresses that are never followed: every call here is refused, or has nothing to do)
AT = 1 << 20


def split_args(**kw):
    a = dict(q=AT, k=AT, v=AT, t=AT, width=8, ctx=AT, qs=AT, n=2, tokens=4, hq=4, hkv=2, d=64, b=16, nb=64,
             scale=0.1, out=AT, work=AT, bytes=1 << 30, dtype=1)
    a.update(kw)
    return [*a.values(), None]


@pytest.mark.parametrize("name", ["pa_decode_drafts", "pa_cross"])
def test_split_attention_refusals(libpa, name):
    f = getattr(libpa.lib(), name)
    for kw in (dict(d=96), dict(b=12), dict(hq=3), dict(hq=258, hkv=2), dict(hkv=0), dict(nb=0), dict(width=0),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(dtype=2),
               dict(dtype=3), dict(n=-1), dict(tokens=-1), dict(hq=65538, hkv=65538),
               dict(q=None), dict(k=None), dict(v=None), dict(t=None), dict(ctx=None), dict(qs=None), dict(out=None),
               dict(q=AT + 2), dict(k=AT + 8), dict(v=AT + 4), dict(out=AT + 1)):
        assert f(*split_args(**kw)) == libpa.PA_ERR_ARG, kw
    for kw in (dict(n=0), dict(tokens=0), dict(n=0, q=None, work=None), dict(tokens=0, out=None)):
        assert f(*split_args(**kw)) == 0, kw
    for heads in ((3, 2, 64), (4, 0, 64), (4, 2, 80), (129, 1, 64)):
        assert libpa.lib().pa_split_workspace_size(*heads) == 0


def rotary_args(**kw):
    a = dict(q=AT, qst=256, k=AT, kst=128, v=AT, vst=128, out=AT, ost=256, kc=AT, vc=AT, t=AT, width=8, ctx=AT, qs=AT,
             f=AT, rd=64, pairs=0, amp=1.0, n=2, tokens=4, nb=64, hq=4, hkv=2, d=64, b=16, dtype=1)
    a.update(kw)
    return a


def test_rotary_refusals(libpa):
    L = libpa.lib()
    common = (dict(rd=24), dict(rd=0), dict(rd=80), dict(rd=-16), dict(amp=math.nan), dict(amp=math.inf), dict(n=-1),
              dict(tokens=-1), dict(d=96), dict(hq=0), dict(hkv=0), dict(dtype=2), dict(dtype=3), dict(q=None),
              dict(k=None), dict(f=None), dict(f=AT + 4), dict(ctx=None), dict(qs=None), dict(out=None),
              dict(qst=255), dict(qst=260), dict(qst=248), dict(kst=120), dict(ost=8), dict(q=AT + 8))
    for kw in common + (dict(kc=None), dict(vc=None), dict(v=None), dict(t=None), dict(vst=64), dict(b=12),
                        dict(nb=0), dict(width=0), dict(kc=AT + 2)):
        assert L.pa_rotary_append(*rotary_args(**kw).values(), None) == libpa.PA_ERR_ARG, kw

    def plain(**kw):
        a = rotary_args(**kw)
        return L.pa_rotary(a["q"], a["qst"], a["k"], a["kst"], a["out"], a["ost"], a["kc"], a["vst"], a["ctx"],
                           a["qs"], a["f"], a["rd"], a["pairs"], a["amp"], a["n"], a["tokens"], a["hq"], a["hkv"],
                           a["d"], a["dtype"], None)
    for kw in common + (dict(kc=None), dict(vst=64), dict(kc=AT + 2)):
        assert plain(**kw) == libpa.PA_ERR_ARG, kw
    for kw in (dict(n=0), dict(tokens=0), dict(n=0, q=None)):
        assert L.pa_rotary_append(*rotary_args(**kw).values(), None) == 0
        assert plain(**kw) == 0


def verify_args(**kw):
    a = dict(tok=AT, p=AT, pst=100, d=AT, dst=100, u=AT, qs=AT, ctx=AT, n=2, tokens=4, V=100, out=AT + 64, em=AT,
             left=AT, dtype=3)
    a.update(kw)
    return [*a.values(), None]


def test_verify_refusals(libpa):
    f = libpa.lib().pa_verify_drafts
    for kw in (dict(V=0), dict(V=2 ** 20 + 1, pst=2 ** 21, dst=2 ** 21), dict(dtype=2), dict(dtype=7), dict(n=-1),
               dict(tokens=-1), dict(pst=99), dict(dst=99), dict(tok=None), dict(p=None), dict(u=None), dict(qs=None),
               dict(ctx=None), dict(out=None), dict(em=None), dict(left=None), dict(out=AT), dict(p=AT + 2),
               dict(d=AT + 1, dtype=0)):
        assert f(*verify_args(**kw)) == libpa.PA_ERR_ARG, kw
    assert f(*verify_args(n=0)) == 0


def test_truncate_gives_blocks_back_in_order(libpa):
    pool = libpa.BlockPool(10, 4)
    pool.allocate(7, 18)  # blocks 0 .. 4
    pool.truncate(7, 18)
    assert pool.block_table(7).tolist() == [0, 1, 2, 3, 4]
    pool.truncate(7, 9)
    assert pool.context_len(7) == 9 and pool.block_table(7).tolist() == [0, 1, 2]
    assert pool.free_list().tolist() == [5, 6, 7, 8, 9, 3, 4]
    assert pool.append_slot(7) == (2 * 4 + 1, None)  # written over the row given up
    pool.truncate(7, 8)
    assert pool.block_table(7).tolist() == [0, 1] and pool.append_slot(7) == (5 * 4, None)
    pool.truncate(7, 0)
    assert pool.block_table(7).tolist() == [] and pool.num_free() == 10
    assert pool.append_slot(7)[0] == 6 * 4


def test_truncate_of_shared_blocks(libpa):
    pool = libpa.BlockPool(10, 4)
    pool.allocate(1, 10)  # blocks 0, 1, 2
    pool.fork(1, 2)
    pool.truncate(2, 5)
    assert [pool.refcount(b) for b in (0, 1, 2)] == [2, 2, 1]
    assert pool.num_free() == 7
    slot, cow = pool.append_slot(2)  # block 1 is shared: copied before the write
    assert cow == (1, 3) and slot == 3 * 4 + 1
    pool.truncate(1, 4)
    assert pool.block_table(1).tolist() == [0] and pool.free_list().tolist() == [4, 5, 6, 7, 8, 9, 1, 2]


def test_truncate_into_a_named_block_forgets_the_name(libpa):
    pool = libpa.BlockPool(10, 4)
    tokens = list(range(12))
    assert pool.allocate_prefix(1, tokens) == 0
    pool.truncate(1, 6)  # block 1 keeps two of its four tokens, block 2 goes back whole
    pool.append_slot(1)  # and takes another token
    assert pool.allocate_prefix(2, tokens) == 4  # the first block alone is what it was
    assert pool.block_table(2)[0] == pool.block_table(1)[0]
    assert pool.block_table(2)[1] != pool.block_table(1)[1]


def test_truncate_refusals(libpa):
    pool = libpa.BlockPool(8, 4, num_cpu_blocks=8)
    pool.allocate(1, 9)
    for n in (-1, 10):
        with pytest.raises(libpa.PagedAttentionError) as e:
            pool.truncate(1, n)
        assert e.value.status == libpa.PA_ERR_ARG
    with pytest.raises(libpa.UnknownSequence):
        pool.truncate(2, 0)
    pool.swap_out([1])
    with pytest.raises(libpa.WrongTier):
        pool.truncate(1, 3)
    assert pool.context_len(1) == 9
