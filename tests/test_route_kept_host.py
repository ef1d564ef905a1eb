"""moe_route_backward_kept answers before anything is launched, as moe_route_backward does."""

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_block_refusals_host import ARG, MISALIGNED, ROUTE, SMALL, UNSUPPORTED, A, _refused  # noqa: E402


def test_refusals():
    for kept in (None, A, A + 1):   # (bytes: any address will do)
        base = ROUTE[:6] + [kept] + ROUTE[6:]
        for changes, code in (({0: None}, ARG), ({5: None}, ARG), ({15: None}, ARG), ({19: None}, ARG), ({1: A + 8}, MISALIGNED),
                              ({5: A + 2}, MISALIGNED), ({7: -1}, ARG), ({8: 192}, UNSUPPORTED), ({10: 17}, UNSUPPORTED),
                              ({20: 64}, SMALL)):
            _refused("moe_route_backward_kept", base, changes, code)
