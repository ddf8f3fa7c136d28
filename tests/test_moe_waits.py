"""The waits of the 64-pair tiles (moe_wide_kernel), read from the built library.

A slab of activations goes from memory straight to LDS, by loads that the
compiler does not count.  Each slab ends in a wait for all of a wave's loads but
the last few, which were issued after the direct ones, and a barrier.  The wait
covers the direct loads only if at least as many ordinary loads as it leaves on
the way stand between the last of them and itself.  That order is the
compiler's work, so it is looked at here, in the library's own code object."""
import os
import re
import struct
import subprocess

import pytest

import ggml_block_quant_amd as ql

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def code_objects(path):
    """The gfx950 code objects of a library: its offload bundles, one a source."""
    data = open(path, "rb").read()
    at = data.find(MAGIC)
    while at >= 0:
        n, = struct.unpack_from("<Q", data, at + len(MAGIC))
        p = at + len(MAGIC) + 8
        for _ in range(n):
            off, size, idlen = struct.unpack_from("<QQQ", data, p)
            p += 24 + idlen
            if b"gfx950" in data[p - idlen:p]:
                yield data[at + off:at + off + size]
        at = data.find(MAGIC, at + 1)


def functions(tmp, name):
    """{symbol: [(address, instruction)]} of the functions whose name holds `name`."""
    out = {}
    for i, obj in enumerate(code_objects(ql.LIB_PATH)):
        if name.encode() not in obj:
            continue
        f = tmp / f"{i}.co"
        f.write_bytes(obj)
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(f)], capture_output=True, text=True, check=True).stdout
        body = None
        for line in text.splitlines():
            m = re.match(r"[0-9a-f]+ <(\S+)>:$", line)
            if m:
                body = out.setdefault(m.group(1), []) if name in m.group(1) else None
            elif body is not None and "//" in line:
                ins, addr = line.split("//", 1)
                target = re.search(r"<\S+?\+0x([0-9a-f]+)>", addr)
                body.append((int(addr.split(":")[0], 16), ins.strip(), int(target.group(1), 16) if target else None))
    return out


def slabs(body):
    """The instructions up to each barrier, since the one before."""
    part = []
    for ins in body:
        part.append(ins)
        if ins[1].startswith("s_barrier"):
            yield part
            part = []


def fault(part, targets=()):
    """What is wrong with a slab's wait, or None.  targets: addresses that a
    branch leads to."""
    direct = [i for i, (_, ins, _) in enumerate(part) if ins.startswith("global_load_lds")]
    if not direct:
        return "no direct load"
    loads = covered = 0
    for addr, ins, _ in part[direct[-1] + 1:]:
        if re.match(r"s_c?branch|s_setpc|s_endpgm", ins) or addr in targets:
            return "a branch between the direct loads and the barrier"
        if re.match(r"(global|buffer|flat|scratch)_load", ins):
            loads += 1
        m = re.search(r"vmcnt\((\d+)\)", ins)
        if m and int(m.group(1)) <= loads:
            covered = 1
    return None if covered else "the wait leaves direct loads on the way"


@pytest.fixture(scope="module")
def wide(tmp_path_factory):
    if not os.path.exists(OBJDUMP):
        pytest.skip("needs llvm-objdump")
    return functions(tmp_path_factory.mktemp("co"), "moe_wide_kernel")


def test_direct_loads_are_waited_for(wide):
    kernels = {k: v for k, v in wide.items() if not k.endswith(".kd")}
    assert len(kernels) == 8  # three formats and Q8_0's ragged rows, two products each
    for name, body in kernels.items():
        start = body[0][0]
        targets = {start + t for _, ins, t in body if t is not None and re.match(r"s_c?branch", ins)}
        parts = list(slabs(body))
        assert len(parts) == 3 and targets, name  # before the loop, and two slabs in it
        for i, part in enumerate(parts):
            assert fault(part, targets) is None, f"{name}, slab {i}: {fault(part, targets)}"


def test_the_check_sees_a_lost_load(wide):
    """Without the ordinary loads behind the direct ones, or with one direct load
    behind them all, every partial wait is found."""
    seen = 0
    for body in wide.values():
        for part in list(slabs(body))[1:]:
            last = max(i for i, (_, ins, _) in enumerate(part) if ins.startswith("global_load_lds"))
            tail = [p for p in part[last + 1:] if not re.match(r"(global|buffer|flat|scratch)_load", p[1]) and "vmcnt(0)" not in p[1]]
            assert fault(part[:last + 1] + tail)
            wait = max(i for i, (_, ins, _) in enumerate(part) if "vmcnt" in ins)
            if "vmcnt(0)" not in part[wait][1]:
                assert fault(part[:wait] + [part[last]] + part[wait:])
                seen += 1
    assert seen >= 8
