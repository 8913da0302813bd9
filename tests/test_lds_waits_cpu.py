"""What the built kernels leave outstanding in LDS where their waves meet, read from the library's own gfx950 code (no GPU).

s_barrier brings the waves of a workgroup together and orders no memory: an LDS write is sure to be seen behind it only if its
wave has waited for it (lgkmcnt).  LDS instructions of a wave finish in order, so on a path through the kernel
a write with k later LDS instructions is done after a wait for lgkmcnt(n), n <= k.  Every path is followed, with the
least k where paths meet.
"""
import os
import re
import struct
import subprocess
from functools import lru_cache

import pytest

import grouped_gemm_expert_offsets_amd as kgw

OBJDUMP = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump")
# labels, kernel names and the instructions that matter; the rest of a line is not looked at
LINE = re.compile(r"^(?:<(?P<label>\w+)>:|\s*(?P<op>ds_\w+|s_waitcnt|s_barrier|s_cbranch\w*|s_branch|s_endpgm)\b[ ]?(?P<args>[^/\n]*))", re.M)
NONE = 1 << 30


def code_objects(path):
    """The gfx950 code objects bundled in a shared library."""
    data, magic = open(path, "rb").read(), b"__CLANG_OFFLOAD_BUNDLE__"
    at = data.find(magic)
    while at >= 0:
        entry = at + 32
        for _ in range(struct.unpack_from("<Q", data, at + 24)[0]):
            offset, size, name = struct.unpack_from("<QQQ", data, entry)
            if size and b"gfx950" in data[entry + 24:entry + 24 + name]:
                yield data[at + offset:at + offset + size]
            entry += 24 + name
        at = data.find(magic, at + 24)


def split(text):
    """{kernel: [(op or None, label or arguments)]} of a disassembly."""
    kernels, body = {}, None
    for m in LINE.finditer(text):
        label = m["label"]
        if label and not re.fullmatch(r"L\d+", label):
            body = kernels.setdefault(label, [])
        elif body is not None:
            body.append((None, label) if label else (m["op"], m["args"].strip()))
    return kernels


@lru_cache(1)
def library(tmp):
    found = {}
    for k, code in enumerate(code_objects(kgw.library_path)):
        path = os.path.join(tmp, f"{k}.o")
        with open(path, "wb") as f:
            f.write(code)
        found.update(split(subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--no-leading-addr", "--symbolize-operands", path],
                                          capture_output=True, text=True, check=True).stdout))
    return found


def outstanding(body, watched):
    """[(place of a barrier, LDS instructions after the watched one)] where one may not be done."""
    blocks, at = [[]], {}
    for place, (op, arg) in enumerate(body):
        if op is None:
            blocks.append([])
            at[arg] = len(blocks) - 1
            continue
        blocks[-1].append((place, op, arg))
        if op.startswith(("s_cbranch", "s_branch", "s_endpgm")):
            blocks.append([])
    after = []
    for k, block in enumerate(blocks):
        op, arg = block[-1][1:] if block else ("", "")
        to = [at[arg]] if op.startswith(("s_cbranch", "s_branch")) else []
        if op not in ("s_branch", "s_endpgm") and k + 1 < len(blocks):
            to.append(k + 1)
        after.append(to)

    def through(k, later, found=None):
        for place, op, arg in blocks[k]:
            if op.startswith("ds_"):
                later = 0 if watched(op) else min(NONE, later + 1)
            elif op == "s_waitcnt":
                n = re.search(r"lgkmcnt\((\d+)\)", arg)
                if n and int(n[1]) <= later:
                    later = NONE
            elif op == "s_barrier" and later < NONE and found is not None:
                found.append((place, later))
        return later

    state, todo = {0: NONE}, [0]
    while todo:
        k = todo.pop()
        later = through(k, state[k])
        for to in after[k]:
            if later < state.get(to, NONE + 1):
                state[to] = later
                todo.append(to)
    found = []
    for k, later in state.items():
        through(k, later, found)
    return sorted(found)


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    if not os.path.exists(OBJDUMP):
        pytest.skip("needs llvm-objdump")
    assert os.path.exists(kgw.library_path), "build the library first"
    return library(str(tmp_path_factory.mktemp("code")))


def test_the_analysis_itself():
    kernel = lambda *lines: split("<k>:\n" + "".join(f"{'' if line[0] == '<' else chr(9)}{line}   // 0\n" for line in lines))["k"]  # noqa: E731
    writes = lambda *lines: outstanding(kernel(*lines), lambda op: "write" in op)  # noqa: E731
    assert writes("ds_write_b32 v0, v1", "s_barrier", "s_endpgm") == [(1, 0)]
    assert not writes("ds_write_b32 v0, v1", "s_waitcnt vmcnt(3) lgkmcnt(0)", "s_barrier", "s_endpgm")
    assert not writes("ds_write_b32 v0, v1", "ds_read_b32 v2, v0", "s_waitcnt lgkmcnt(1)", "s_barrier", "s_endpgm")
    assert writes("ds_write_b32 v0, v1", "ds_read_b32 v2, v0", "s_waitcnt lgkmcnt(2)", "s_barrier", "s_endpgm") == [(3, 1)]
    # the wait is on one of two paths only
    assert writes("ds_write_b32 v0, v1", "s_cbranch_execz L0", "s_waitcnt lgkmcnt(0)", "<L0>:", "s_barrier", "s_endpgm") == [(4, 0)]
    # a write at the end of a loop meets the barrier at its start
    assert writes("<L0>:", "s_barrier", "ds_write_b32 v0, v1", "s_cbranch_scc0 L0", "s_endpgm") == [(1, 0)]


def test_the_claimed_item_is_passed_on_through_lds(kernels):
    """The kernels whose workgroups claim their tiles pass an item on in one 32-bit word of LDS, the only one that they use."""
    claiming = {k: v for k, v in kernels.items() if "wgrad_bf16_kernel" in k or "wgrad_rows8_kernel" in k}
    assert len(claiming) >= 30
    for name, body in claiming.items():
        assert any(op == "ds_write_b32" for op, _ in body), name
        assert not outstanding(body, lambda op: op == "ds_write_b32"), name
        assert not outstanding(body, lambda op: op == "ds_read_b32"), name


def test_no_write_is_outstanding_where_waves_meet(kernels):
    """Not the results staged by a wave that stores none of them (its part of a tile lies outside the matrix) either: the
    next tile's operands go to the same place."""
    assert sum("wgrad" in k or "mgrouped" in k for k in kernels) >= 70
    bad = [k for k, body in kernels.items() if outstanding(body, lambda op: "write" in op or op.startswith("ds_add"))]
    assert not bad, f"{len(bad)} kernels, first {bad[:3]}"
