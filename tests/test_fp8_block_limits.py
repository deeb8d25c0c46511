"""Limits of the FP8 block-scale calls on the host: head counts past 32-bit offsets are refused."""
P = 1 << 20  # an aligned address that no refused call dereferences


def test_prefill_refuses_heads_past_its_offsets(libpa):
    args = lambda hq, hkv, n: (P, P, P, P, P, P, 4, P, P, n, 20, 9, hq, hkv, 128, 16, 8, 0.1, P, 1, None)  # noqa: E731
    run = libpa.lib().pa_prefill_fp8_block
    assert run(*args(1 << 17, 1 << 17, 3)) == libpa.PA_ERR_ARG
    assert run(*args(1 << 17, 1 << 17, 0)) == libpa.PA_ERR_ARG
    assert run(*args(65536, 65536, 0)) == libpa.PA_OK  # (no sequences)
