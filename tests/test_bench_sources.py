"""The sources that bench.py's stored HBM traffic is keyed to: the block's
forward pass, and nothing beside it."""
import os

import bench


def test_key_covers_the_forward_pass_alone():
    names = {os.path.basename(p) for p in bench.KERNEL_SOURCES}
    assert {"route.hip", "permute.hip", "ffn.hip", "combine.hip", "moe_api.hip", "common.h", "kernels.h",
            "tiles.h", "schedule.h"} <= names
    # the products by themselves, their gradients and the int8 experts
    assert not names & {"grouped.hip", "gemm_tile.h", "gemm_wgrad.h", "swiglu.hip", "codes.h", "peak.hip"}
    assert bench.OTHER_SOURCES <= set(os.listdir(os.path.join(bench.ROOT, "group_limited_routing_router_amd",
                                                              "csrc")))


def test_other_sources_are_not_included_by_the_forward_pass():
    for rel in bench.KERNEL_SOURCES:
        with open(os.path.join(bench.ROOT, rel)) as f:
            text = f.read()
        assert not [n for n in bench.OTHER_SOURCES if f'#include "{n}"' in text], rel
