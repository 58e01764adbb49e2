"""Registers of the compiled kernels, from the metadata of the code objects in the built library: a matrix-product kernel
whose loop runs out of vector registers reloads them from scratch memory between its MFMAs, and each reload waits for
the tiles on their way from memory as well.  The results stay right, so nothing else would tell."""

import functools
import os
import re
import shutil
import struct
import subprocess

import pytest

import fp8_blockwise_quantized_amd as fq
from fp8_blockwise_quantized_amd import build

MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def _readelf():
    beside = os.path.join(os.path.dirname(os.path.realpath(build.HIPCC)), "..", "llvm", "bin", "llvm-readelf")
    for path in (beside, "/opt/rocm/llvm/bin/llvm-readelf", shutil.which("llvm-readelf")):
        if path and os.path.exists(path):
            return path
    pytest.skip("llvm-readelf not available")


@functools.lru_cache(maxsize=None)
def kernels(folder):
    """(name, template arguments, vector registers spilled, bytes of scratch) of every gfx950 kernel of the library."""
    data = open(fq.LIB_PATH, "rb").read()
    found, at = [], data.find(MAGIC)
    while at >= 0:  # one bundle per source file: a count, then offset, size and target of each entry
        p = at + len(MAGIC) + 8
        for _ in range(struct.unpack_from("<Q", data, p - 8)[0]):
            offset, size, n = struct.unpack_from("<QQQ", data, p)
            target = data[p + 24:p + 24 + n]
            p += 24 + n
            if b"gfx950" not in target or size == 0:
                continue
            path = os.path.join(folder, f"{at}.o")
            with open(path, "wb") as f:
                f.write(data[at + offset:at + offset + size])
            notes = subprocess.run([_readelf(), "--notes", path], capture_output=True, text=True, check=True).stdout
            for k in notes.split(".agpr_count")[1:]:
                symbol = re.search(r"\.symbol:\s+(\S+)", k).group(1)
                spilled, scratch = (int(re.search(rf"\.{f}:\s+(\d+)", k).group(1))
                                    for f in ("vgpr_spill_count", "private_segment_fixed_size"))
                n, rest = re.match(r"_ZN5fp8bqL?(\d+)(.*)", symbol).groups()  # (mangled: length, name, arguments)
                args = re.match(r"I(?:[a-z]|L[a-z]\d+E)+E", rest[int(n):])
                found.append((rest[:int(n)], [int(v) for v in re.findall(r"L[a-z](\d+)E", args.group(0))] if args else [],
                              spilled, scratch))
        at = data.find(MAGIC, at + 1)
    return found


@pytest.fixture
def all_kernels(tmp_path_factory):
    return kernels(str(tmp_path_factory.getbasetemp()))


def test_grouped_weight_gradient_added_to_the_output(all_kernels):
    """The form a training loop with FP32 main gradients takes (4 format pairs, 3 tile shapes)."""
    mine = [k for k in all_kernels if k[0] == "gemm_tn_kernel" and k[1][0] == 2 and k[1][-2:] == [2, 3]]
    assert len(mine) == 12
    assert [k for k in mine if k[2] or k[3]] == []
