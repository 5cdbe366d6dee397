"""The compiled tiles of the FP8 products and of the weight gradient, as built in
libmoe.so: no spilled registers, no scratch memory, and no lane mask behind the
last matrix instruction.

On the 256-row tiles nearly all 512 registers hold sums or the gradient of h. A
value that the compiler moves inside a lane mask, because registers run out
there, is lost in the other lanes: the gradients of experts whose last block
of 32 rows is not full came out wrong that way, with no error anywhere."""
import os
import re
import struct
import subprocess

import pytest

from group_limited_routing_router_amd import moe

LLVM = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin")
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"
# and how many there are: products of three tiles, gathered or not, with and
# without weights past the caches; input gradients, not gathered; the gated pass
# as the products, twice; weight gradients of two tiles, gathered or not, bf16,
# fp32 and added to
KERNELS = {"fp8_tile_kernel": 10 + 5 + 2 * 10, "gemm_wgrad_kernel": 2 * 2 * 3}


def code_objects():
    """The gfx950 code objects of libmoe.so, one for each source."""
    with open(moe.library_path(), "rb") as f:
        data = f.read()
    at = data.find(MAGIC)
    while at >= 0:
        (n,) = struct.unpack_from("<Q", data, at + len(MAGIC))
        entry = at + len(MAGIC) + 8
        for _ in range(n):
            offset, size, length = struct.unpack_from("<QQQ", data, entry)
            target = data[entry + 24:entry + 24 + length]
            entry += 24 + length
            if b"gfx950" in target and size:
                yield data[at + offset:at + offset + size]
        at = data.find(MAGIC, at + len(MAGIC))


@pytest.fixture(scope="module")
def tiles(tmp_path_factory):
    """Kernel -> (its numbers in the metadata, its instructions)."""
    d = tmp_path_factory.mktemp("code")
    got = {}
    for i, code in enumerate(code_objects()):
        if not any(k.encode() in code for k in KERNELS):
            continue
        path = d / f"{i}.co"
        path.write_bytes(code)
        notes = subprocess.run([os.path.join(LLVM, "llvm-readelf"), "--notes", str(path)], check=True,
                               capture_output=True, text=True).stdout
        numbers = {}
        for block in notes.split("  - .agpr_count:")[1:]:
            name = re.search(r"\.name:\s+(\S+)", block).group(1)
            numbers[name] = {k: int(v) for k, v in re.findall(r"\.(\w+):\s+(\d+)\n", ".agpr_count:" + block)}
        text = subprocess.run([os.path.join(LLVM, "llvm-objdump"), "-d", "--no-show-raw-insn", "--mcpu=gfx950",
                               str(path)], check=True, capture_output=True, text=True).stdout
        for part in re.split(r"\n(?=[0-9a-f]+ <)", text):
            m = re.match(r"[0-9a-f]+ <(\S+)>:\n", part)
            if m and any(k in m.group(1) for k in KERNELS):
                got[m.group(1)] = numbers[m.group(1)], [x.split("//")[0].strip() for x in part.splitlines()[1:]]
    assert all(sum(k in name for name in got) == n for k, n in KERNELS.items()), sorted(got)
    return got


def test_no_spills_and_no_scratch(tiles):
    bad = {n: (v["vgpr_spill_count"], v["private_segment_fixed_size"]) for n, (v, _) in tiles.items()
           if v["vgpr_spill_count"] or v["private_segment_fixed_size"]}
    assert not bad, bad


def writes_mask(line):
    return "saveexec" in line or re.match(r"(s_\w+|v_cmpx\w+) exec(_lo|_hi)?\b", line) is not None


def test_no_lane_mask_behind_the_sums(tiles):
    bad = {}
    for name, (_, code) in tiles.items():
        last = max(i for i, x in enumerate(code) if x.startswith("v_mfma"))
        assert any(writes_mask(x) for x in code[:last])  # the schedule's, so they are found
        found = [x for x in code[last:] if writes_mask(x)]
        if found:
            bad[name] = len(found)
    assert not bad, bad
