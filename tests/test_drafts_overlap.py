"""Outputs that lie over inputs, refused before any CUDA call."""
from test_drafts_host import AT, rotary_args, verify_args


def test_verify_outputs_over_inputs(libpa):
    """A sequence's tokens, or another sequence's length, would be written while they are read."""
    f = libpa.lib().pa_verify_drafts
    far = AT + 4096
    for off in (-12, -4, 0, 4, 12):  # of four tokens
        assert f(*verify_args(tok=far, out=far + off)) == libpa.PA_ERR_ARG, off
    for off in (-4, 4):  # of two lengths
        assert f(*verify_args(ctx=far, left=far + off)) == libpa.PA_ERR_ARG, off


def test_rows_in_place_keep_their_places(libpa):
    L = libpa.lib()
    for kw in (dict(ost=512), dict(qst=264)):
        assert L.pa_rotary_append(*rotary_args(**kw).values(), None) == libpa.PA_ERR_ARG, kw
    for q, k in ((256, 136), (264, 128)):  # q_out is q and key_out is key; rows of 256 and 128 values
        assert L.pa_rotary(AT, q, 2 * AT, k, AT, 256, 2 * AT, 128, AT, AT, AT, 64, 0, 1.0, 2, 4, 4, 2, 64, 1,
                           None) == libpa.PA_ERR_ARG, (q, k)
