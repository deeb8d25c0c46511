"""Outputs that lie over inputs, refused before any CUDA call."""
from test_drafts_host import AT, verify_args


def test_verify_outputs_over_inputs(libpa):
    """A sequence's tokens, or another sequence's length, would be written while they are read."""
    f = libpa.lib().pa_verify_drafts
    far = AT + 4096
    for off in (-12, -4, 0, 4, 12):  # of four tokens
        assert f(*verify_args(tok=far, out=far + off)) == libpa.PA_ERR_ARG, off
    for off in (-4, 4):  # of two lengths
        assert f(*verify_args(ctx=far, left=far + off)) == libpa.PA_ERR_ARG, off
