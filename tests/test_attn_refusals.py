"""Calls of the attention layers that are refused before any launch, beside those of test_attn_host.py."""
import pytest

from test_attn_host import A, INVALID, backward, lib  # noqa: F401


@pytest.mark.parametrize("grad,ld,hs,dense", [("dq", "ld_dq", "hs_dq", (1024, 128)), ("dk", "ld_dk", "hs_dk", (256, 128))])
def test_gradients_in_place_have_the_place_s_layout(lib, grad, ld, hs, dense):  # noqa: F811
    """dq in dq_out's memory, with any other distances, would overwrite gradients that are still to be read."""
    src = grad + "_out"
    for layout in ((dense[0] + 512, dense[1]), (dense[0] * 2, dense[1] * 2), (dense[1], dense[1] * 6)):
        assert backward(lib, **{grad: A, src: A, ld: layout[0], hs: layout[1]}) == INVALID, layout
