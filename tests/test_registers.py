"""What the compiler made of the kernels, from the code objects in the built library, where the results stay right and
nothing else would tell.  Registers, from the metadata: a matrix-product kernel whose loop runs out of vector registers
reloads them from scratch memory between its MFMAs, and each reload waits for the tiles on their way from memory as
well.  Stores: a branch with the same store on both sides, cached on one and past the caches on the other, is one the
compiler likes to fold into a single cached store."""

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


def _tool(name):
    beside = os.path.join(os.path.dirname(os.path.realpath(build.HIPCC)), "..", "llvm", "bin", name)
    for path in (beside, os.path.join("/opt/rocm/llvm/bin", name), shutil.which(name)):
        if path and os.path.exists(path):
            return path
    pytest.skip(f"{name} not available")


def _kernel(symbol):
    """Name and template arguments (those that are numbers) of a mangled kernel."""
    n, rest = re.match(r"_ZN5fp8bqL?(\d+)(.*)", symbol).groups()  # (mangled: length, name, arguments)
    args = re.match(r"I(?:[a-z]|L[a-z]\d+E)+E", rest[int(n):])
    return rest[:int(n)], [int(v) for v in re.findall(r"L[a-z](\d+)E", args.group(0))] if args else []


@functools.lru_cache(maxsize=None)
def code_objects(folder):
    """Files with the library's gfx950 code objects, one of each source file."""
    data = open(fq.LIB_PATH, "rb").read()
    files, at = [], data.find(MAGIC)
    while at >= 0:  # one bundle per source file: a count, then offset, size and target of each entry
        p = at + len(MAGIC) + 8
        for _ in range(struct.unpack_from("<Q", data, p - 8)[0]):
            offset, size, n = struct.unpack_from("<QQQ", data, p)
            target = data[p + 24:p + 24 + n]
            p += 24 + n
            if b"gfx950" not in target or size == 0:
                continue
            files.append(os.path.join(folder, f"{at}.o"))
            with open(files[-1], "wb") as f:
                f.write(data[at + offset:at + offset + size])
        at = data.find(MAGIC, at + 1)
    return files


@functools.lru_cache(maxsize=None)
def kernels(folder):
    """(name, template arguments, vector registers spilled, bytes of scratch) of every kernel of the library."""
    found = []
    for path in code_objects(folder):
        notes = subprocess.run([_tool("llvm-readelf"), "--notes", path], capture_output=True, text=True, check=True).stdout
        for k in notes.split(".agpr_count")[1:]:
            symbol = re.search(r"\.symbol:\s+(\S+)", k).group(1)
            found.append((*_kernel(symbol), *(int(re.search(rf"\.{f}:\s+(\d+)", k).group(1))
                                              for f in ("vgpr_spill_count", "private_segment_fixed_size"))))
    return found


@pytest.fixture
def folder(tmp_path_factory):
    return str(tmp_path_factory.getbasetemp())


@pytest.fixture
def all_kernels(folder):
    return kernels(folder)


def test_grouped_weight_gradient_added_to_the_output(all_kernels):
    """The form a training loop with FP32 main gradients takes (4 format pairs, 3 tile shapes)."""
    mine = [k for k in all_kernels if k[0] == "gemm_tn_kernel" and k[1][0] == 2 and k[1][-2:] == [2, 3]]
    assert len(mine) == 12
    assert [k for k in mine if k[2] or k[3]] == []


def test_no_kernel_spills(all_kernels):
    assert len(all_kernels) > 300
    assert [k for k in all_kernels if k[2] or k[3]] == []


def test_both_kinds_of_store(folder):
    """Every product kernel that stores whole lines of full tiles can store them past the caches and not: fprop and dgrad in
    BF16, wgrad and the MXFP4 products in BF16 and FP32 (the 64-row MXFP4 tile in FP32 only)."""
    expect = set()
    for path in code_objects(folder):
        text = subprocess.run([_tool("llvm-objdump"), "-d", path], capture_output=True, text=True, check=True).stdout
        for body in re.split(r"\n(?=[0-9a-f]{16} <)", text):
            symbol = re.match(r"[0-9a-f]{16} <(_ZN5fp8bq\S+)>", body)
            name, args = _kernel(symbol.group(1)) if symbol else ("", [])
            if name == "gemm_tn_kernel":
                lines = args[9] == 0 or (args[0] == 2 and args[9] == 1)
            elif name == "gemm_tn_grouped_kernel":
                lines = args[4] == 0
            elif name == "mx_gemm_kernel":
                lines = (args[0] >= 128 and args[6] == 0) or args[6] == 1
            else:
                continue
            wide = re.findall(r"global_store_dwordx4 [^/]*", body)
            past = sum(" nt" in w for w in wide)
            if lines:
                expect.add(name)
                assert past > 0 and len(wide) - past >= past, (name, args)
            else:
                assert past == 0, (name, args)
    assert expect == {"gemm_tn_kernel", "gemm_tn_grouped_kernel", "mx_gemm_kernel"}
