"""CPU check of the hand-written LDS-DMA sequences in the kernel sources.

A load to LDS takes its LDS address from m0, and the hardware needs one wait
state between a scalar write of m0 and such a load.  The compiler inserts it for
code of its own but does not look into an asm string."""
import glob
import os
import re
import shutil
import struct
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "contextual_sparsity_lora_svd_amd", "csrc")


def _asm_strings():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.h*"))):
        text = open(path).read()
        for m in re.finditer(r'asm(?:\s+volatile)?\s*\(\s*((?:"(?:[^"\\]|\\.)*"\s*)+)', text):
            body = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', m.group(1)))
            yield f"{os.path.basename(path)}:{text.count(chr(10), 0, m.start()) + 1}", body


def test_a_wait_state_stands_between_m0_and_the_load_to_lds():
    found, missing = 0, []
    for where, body in _asm_strings():
        written = False                       # m0 written by the instruction before
        for ins in re.split(r"\\n(?:\\t)?|;", body):
            ins = ins.strip()
            if re.search(r"\bload_lds\b|_load_lds_", ins):
                found += 1
                if written:
                    missing.append(where)
            written = bool(re.match(r"s_\w+\s+m0\b", ins))
    assert found >= 6
    assert not missing, f"no wait state after m0 is written: {missing}"


def _code_objects(path):
    """The gfx950 code objects bundled in a shared library built by hipcc."""
    blob, magic, at = open(path, "rb").read(), b"__CLANG_OFFLOAD_BUNDLE__", 0
    while (at := blob.find(magic, at)) >= 0:
        pos = at + len(magic)
        (count,) = struct.unpack_from("<Q", blob, pos)
        pos += 8
        for _ in range(count):
            off, size, n = struct.unpack_from("<QQQ", blob, pos)
            triple = blob[pos + 24:pos + 24 + n]
            pos += 24 + n
            if triple.endswith(b"gfx950") and size:
                yield blob[at + off:at + off + size]
        at += len(magic)


def _sgprs(operand):
    m = re.match(r"s\[(\d+):(\d+)\]|s(\d+)\b", operand)
    if not m:
        return set()
    return {int(m[3])} if m[3] else set(range(int(m[1]), int(m[2]) + 1))


def _short_waits(listing):
    """Loads to LDS whose m0 was written by the instruction before, or whose scalar
    base a vector instruction wrote fewer than 5 wait states before."""
    vector, m0, found, short = {}, 99, 0, []
    for line in listing.splitlines():
        m = re.match(r"\s+([a-z]\w+)(?:\s+(.*?))?\s*(?://.*)?$", line)
        if not m:
            continue
        op, ops = m[1], [x.strip() for x in (m[2] or "").split(",")]
        if "load_lds" in op:
            found += 1
            base = set().union(*(_sgprs(x) for x in ops))
            if m0 < 1 or any(vector.get(r, 99) < 5 for r in base):
                short.append(line.strip())
        states = int(ops[0]) + 1 if op == "s_nop" else 1
        vector = {r: n + states for r, n in vector.items() if n + states < 5}
        m0 += states
        if ops[0] == "m0":
            m0 = 0
        written = _sgprs(ops[0])
        if op.startswith("v_"):
            if len(ops) > 1 and re.match(r"v_(add|sub|subrev|addc|subb)_co|v_mad_[ui]64|v_div_scale", op):
                written |= _sgprs(ops[1])
            vector.update({r: 0 for r in written})
        else:
            for r in written:
                vector.pop(r, None)
    return found, short


def test_waits_of_the_built_kernels(tmp_path):
    """The same in the library as it was built, and the wait the hardware needs
    between a vector write of the scalar base and the load (which the source
    cannot show: the compiler places what computes the base)."""
    from contextual_sparsity_lora_svd_amd import build
    objdump = shutil.which("llvm-objdump") or "/opt/rocm/llvm/bin/llvm-objdump"
    if not os.path.exists(objdump):
        pytest.skip("no llvm-objdump")
    if not os.path.exists(build.LIB):
        build.build(verbose=False)
    total = 0
    for i, code in enumerate(_code_objects(build.LIB)):
        obj = tmp_path / f"{i}.co"
        obj.write_bytes(code)
        text = subprocess.run([objdump, "-d", "--no-show-raw-insn", str(obj)], capture_output=True, text=True,
                              check=True).stdout
        found, short = _short_waits(text)
        total += found
        assert not short, (i, len(short), short[:4])
    assert total > 500
