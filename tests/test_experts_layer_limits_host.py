"""The sizes that include/expert_layer.h allows the few-token layer are those that
its workspace size is given for and its call accepts (CPU only: a call is made
just past each limit, where it is refused)."""
import os
import re

import pytest

from test_feed_forward_abi_host import call, lib  # noqa: F401

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "expert_layer.h")


def limits():
    text = open(HEADER).read()
    layer = text[text.index("A whole expert layer for a few tokens"):]
    m = re.search(r"T <= (\d+), T \* k <= (\d+), H and F <= (\d+)", layer)
    assert m, "the header states the layer's limits"
    return tuple(int(x) for x in m.groups())


def test_sizes_up_to_the_stated_limits_are_accepted(lib):  # noqa: F811
    T, S, side = limits()
    for t, k, H, F in ((T, S // T, 64, 64), (T, 1, 64, 64), (S // 64, 64, 64, 64), (1, 64, 64, 64),
                       (1, 1, side, side), (T, S // T, side, side)):
        assert lib.sgemm_experts_layer_workspace_size(t, k, H, F) == t * k * -(-F // 16) * 16 * 4


@pytest.mark.parametrize("which", ["T", "T * k", "H", "F"])
def test_sizes_past_them_are_refused(lib, which):  # noqa: F811
    T, S, side = limits()
    t, k, H, F = {"T": (T + 1, 1, 64, 64), "T * k": (T, S // T + 1, 64, 64),
                  "H": (1, 1, side + 16, 64), "F": (1, 1, 64, side + 16)}[which]
    assert lib.sgemm_experts_layer_workspace_size(t, k, H, F) == 0
    assert call(lib, "sgemm_experts_layer", T=t, k=k, H=H, F=F, ldx=H, ldo=H, ld1=H, ld2=F,
                stride1=2 * F * H, stride2=H * F,
                workspace_bytes=1 << 40) == lib.SGEMM_ERR_INVALID_ARG
