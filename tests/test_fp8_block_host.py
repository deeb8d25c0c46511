"""Refusals of the FP8 block-scale calls and of build_step, on the host: shapes, types, null and
misaligned pointers are rejected before anything is launched, and a planned launch holds its
tensors."""
import gc

import pytest
import torch

N, HQ, HKV, D, NB, B, T = 3, 8, 2, 64, 8, 16, 4
P = 1 << 20  # an aligned address that no refused call dereferences


def build_args(**kw):
    a = dict(q=P, c=P, n=N, free=P, nfree=NB, start=P, tables=P, T=T, B=B, nb=NB, slots=P, ns=9,
             qs=P, nxt=P + 16)
    a.update(kw)
    return (*a.values(), None)


@pytest.mark.parametrize("bad", [dict(B=12), dict(nb=0), dict(T=0), dict(n=-1), dict(nfree=-1),
                                 dict(ns=-1), dict(nxt=P), dict(start=None), dict(nxt=None),
                                 dict(qs=None), dict(q=None), dict(c=None), dict(tables=None),
                                 dict(slots=None), dict(free=None), dict(T=1 << 28)])
def test_build_step_refusals(libpa, bad):
    assert libpa.lib().pa_build_step(*build_args(**bad)) == libpa.PA_ERR_ARG


def append_args(**kw):
    a = dict(key=P, value=P, kc=P, vc=P, ks=P, vs=P, tables=P, T=T, c=P, qs=P, n=N, rows=9, nb=NB,
             hkv=HKV, d=D, B=B, dtype=1)
    a.update(kw)
    return (*a.values(), None)


@pytest.mark.parametrize("bad", [dict(d=96), dict(B=12), dict(hkv=0), dict(nb=0), dict(T=0),
                                 dict(n=-1), dict(rows=-1), dict(dtype=2), dict(key=None),
                                 dict(value=P + 8), dict(kc=P + 8), dict(vs=P + 2), dict(ks=None),
                                 dict(tables=None), dict(c=None), dict(qs=None), dict(T=1 << 28),
                                 dict(nb=1 << 27)])
def test_append_refusals(libpa, bad):
    assert libpa.lib().pa_append_fp8_block(*append_args(**bad)) == libpa.PA_ERR_ARG


def test_append_of_nothing(libpa):
    assert libpa.lib().pa_append_fp8_block(*append_args(n=0, key=None)) == libpa.PA_OK
    assert libpa.lib().pa_append_fp8_block(*append_args(rows=0, key=None)) == libpa.PA_OK


def decode_args(**kw):
    a = dict(q=P, kc=P, vc=P, ks=P, vs=P, tables=P, T=T, c=P, n=N, hq=HQ, hkv=HKV, d=D, B=B, nb=NB,
             scale=0.1, out=P, ws=P, wsb=1 << 30, dtype=1)
    a.update(kw)
    return (*a.values(), None)


BAD_ATTENTION = [dict(d=96), dict(B=12), dict(hq=7), dict(hkv=0), dict(nb=0), dict(T=0), dict(n=-1),
                 dict(scale=float("nan")), dict(dtype=2), dict(q=None), dict(q=P + 8), dict(kc=None),
                 dict(vc=P + 8), dict(ks=None), dict(vs=P + 1), dict(tables=None), dict(c=None),
                 dict(out=None), dict(out=P + 8)]


@pytest.mark.parametrize("bad", BAD_ATTENTION)
def test_decode_refusals(libpa, bad):
    assert libpa.lib().pa_decode_fp8_block(*decode_args(**bad)) == libpa.PA_ERR_ARG


@pytest.mark.parametrize("bad", BAD_ATTENTION + [dict(most=-1), dict(rows=-1), dict(qs=None),
                                                 dict(hq=130), dict(scale=0.0), dict(scale=-0.1)])
def test_prefill_refusals(libpa, bad):
    a = dict(q=P, kc=P, vc=P, ks=P, vs=P, tables=P, T=T, c=P, qs=P, n=N, rows=20, most=9, hq=HQ, hkv=HKV, d=D,
             B=B, nb=NB, scale=0.1, out=P, dtype=1)
    a.update(bad)
    assert libpa.lib().pa_prefill_fp8_block(*a.values(), None) == libpa.PA_ERR_ARG


def test_copy_and_swap_refusals(libpa):
    lib = libpa.lib()
    for bad in (dict(d=96), dict(B=9), dict(n=-1), dict(nb=0), dict(kc=None), dict(ks=None),
                dict(vc=P + 8), dict(vs=P + 2), dict(m=None)):
        a = dict(kc=P, vc=P, ks=P, vs=P, m=P, n=2, nb=NB, hkv=HKV, d=D, B=B)
        a.update(bad)
        assert lib.pa_copy_blocks_fp8_block(*a.values(), None) == libpa.PA_ERR_ARG, bad
    for bad in (dict(d=96), dict(n=-1), dict(nbs=0), dict(nbd=0)):
        a = dict(a=P, b=P, c=P, d_=P, e=P, f=P, g=P, h=P, m=P, n=2, nbs=NB, nbd=NB, hkv=HKV, d=D, B=B)
        a.update(bad)
        assert lib.pa_swap_blocks_fp8_block(*a.values(), None) == libpa.PA_ERR_ARG, bad
    assert lib.pa_copy_blocks_fp8_block(None, None, None, None, None, 0, NB, HKV, D, B, None) == 0


@pytest.fixture
def cpu_marshal(libpa, monkeypatch):
    """CPU tensors pass for those of device -1: marshalling without a GPU."""
    monkeypatch.setattr(libpa, "_device_of", lambda t, name: -1)
    monkeypatch.setattr(libpa, "make_workspace", lambda *a: torch.empty(256, dtype=torch.uint8))
    return libpa


def cache():
    return (torch.zeros(NB, HKV, B, D, dtype=torch.uint8), torch.zeros(NB, HKV, B, D, dtype=torch.uint8),
            torch.ones(NB, HKV), torch.ones(NB, HKV))


def test_planned_launches_hold_their_tensors(cpu_marshal):
    pa = cpu_marshal
    i32 = dict(dtype=torch.int32)
    tables, lens, qs = torch.zeros(N, T, **i32), torch.ones(N, **i32), torch.zeros(N + 1, **i32)
    rows = torch.zeros(N, HKV, D, dtype=torch.bfloat16)
    q = torch.zeros(N, HQ, D, dtype=torch.bfloat16)
    made = [pa.append_fp8_block(rows, rows.clone(), *cache(), tables, lens, qs, plan=True),
            pa.decode_fp8_block(q, *cache(), tables, lens, 0.1, plan=True),
            pa.prefill_fp8_block(q, *cache(), tables, lens, qs, 0.1, 1, plan=True),
            pa.build_step(lens, lens.clone(), torch.zeros(NB, **i32), torch.zeros(1, **i32), tables, B,
                          NB, torch.zeros(9, dtype=torch.int64), qs, torch.zeros(1, **i32), plan=True)]
    for launch in made:
        gc.collect()
        held = {t.data_ptr() for t in (*launch._keep, launch.out)}
        pointers = [a for a in launch._args if isinstance(a, int) and a > 1 << 16]
        assert pointers and set(pointers) <= held, launch._name
    with pytest.raises(ValueError, match="planned build_step needs"):
        pa.build_step(lens, lens, tables[0], lens[:1], tables, B, NB, qs.long(), plan=True)


def test_shape_and_type_checks_name_the_argument(cpu_marshal):
    pa = cpu_marshal
    kc, vc, ks, vs = cache()
    tables, lens = torch.zeros(N, T, dtype=torch.int32), torch.ones(N, dtype=torch.int32)
    q = torch.zeros(N, HQ, D, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match=r"scales \[NB, Hkv\]"):
        pa.decode_fp8_block(q, kc, vc, ks[:, :1], vs, tables, lens, 0.1)
    with pytest.raises(ValueError, match="k_cache must be a CUDA tensor"):
        pa.decode_fp8_block(q, kc.float(), vc, ks, vs, tables, lens, 0.1)
    with pytest.raises(ValueError, match="tables must be a CUDA tensor"):
        pa.decode_fp8_block(q, kc, vc, ks, vs, tables.long(), lens, 0.1)
    with pytest.raises(ValueError, match="out must match q"):
        pa.decode_fp8_block(q, kc, vc, ks, vs, tables, lens, 0.1, out=q.float())
    rows = torch.zeros(N, HKV, D, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="query_start must be"):
        pa.append_fp8_block(rows, rows, kc, vc, ks, vs, tables, lens, lens)
    start = torch.zeros(N + 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="value must be"):
        pa.append_fp8_block(rows, rows.half(), kc, vc, ks, vs, tables, lens, start)
    with pytest.raises(ValueError, match="value must be"):
        pa.append_fp8_block(rows, rows.transpose(0, 1).contiguous().transpose(0, 1), kc, vc, ks, vs,
                            tables, lens, start)
    with pytest.raises(TypeError, match="unsupported dtype"):
        pa.append_fp8_block(rows.float(), rows.float(), kc, vc, ks, vs, tables, lens, start)


def test_tensors_of_another_device_are_refused(libpa):
    """Every tensor must be on the device of the call's first one, and that a CUDA device."""
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        libpa.decode_fp8_block(torch.zeros(N, HQ, D, dtype=torch.float16), *cache(),
                               torch.zeros(N, T, dtype=torch.int32), torch.ones(N, dtype=torch.int32), 0.1)

    class On:
        def __init__(self, dev, dtype=torch.int32):
            self.dev, self.dtype, self.is_cuda = dev, dtype, dev >= 0

        def get_device(self):
            return self.dev

        def is_contiguous(self):
            return True

        def data_ptr(self):
            return P

    assert libpa._ptr(On(1), "lens", torch.int32, 1) == P
    assert libpa._codes_ptr(On(0, torch.uint8), "k_cache", 0) == P
    for t, match in ((On(0), "another device"), (On(-1), "CUDA tensor"), (On(1, torch.int64), "must be torch.int32, got")):
        with pytest.raises(ValueError, match=match):
            libpa._ptr(t, "lens", torch.int32, 1)
    with pytest.raises(ValueError, match="uint8 or torch.float8_e4m3fn, got"):
        libpa._codes_ptr(On(1, torch.float16), "k_cache", 1)


def test_calls_make_their_tensors_device_current(libpa):
    for name in ("build_step", "append_fp8_block", "decode_fp8_block", "prefill_fp8_block",
                 "copy_blocks_fp8_block",
                 "swap_blocks_fp8_block"):
        assert hasattr(getattr(libpa, name), "__wrapped__"), name
