"""The kernels inside the built library, as the compiler describes them: their notes (registers, scratch, LDS) and their code."""
import os
import re
import struct
import subprocess

import pytest

from token_dispatch_expert_amd import binding as B

TOOLS = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin")
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def tool(name):
    path = os.path.join(TOOLS, name)
    if not os.path.exists(path):
        pytest.skip(f"needs {path}")
    return path


def unbundle(folder):
    """The device code objects of the library, one for each source file, as files in `folder`."""
    if not os.path.exists(B.library_path()):
        pytest.fail("library missing: run __graft_entry__.build()")
    with open(B.library_path(), "rb") as f:
        data = f.read()
    files = []
    for m in re.finditer(re.escape(MAGIC), data):
        at = m.end()
        count, = struct.unpack_from("<Q", data, at)
        at += 8
        for _ in range(count):
            offset, size, length = struct.unpack_from("<QQQ", data, at)
            name = data[at + 24:at + 24 + length].decode()
            at += 24 + length
            if "gfx950" in name and size:
                path = os.path.join(folder, f"{len(files)}.o")
                with open(path, "wb") as f:
                    f.write(data[m.start() + offset:m.start() + offset + size])
                files.append(path)
    assert files, "no device code found"
    return files


def notes(files):
    """symbol -> {field: number} of every kernel."""
    kernels = {}
    for path in files:
        text = subprocess.run([tool("llvm-readelf"), "--notes", path], capture_output=True, text=True, check=True).stdout
        for entry in re.split(r"\n  - (?=\.agpr_count|\.args)", text)[1:]:
            name = re.search(r"^ +\.name: +(\S+)", entry, re.M)
            fields = dict(re.findall(r"^ *\.(\w+): +(\d+)$", entry, re.M))
            kernels[name[1]] = {k: int(v) for k, v in fields.items()}
    return kernels


def code(files, containing):
    """symbol -> instructions (one a line) of every kernel whose name contains the text."""
    found = {}
    for path in files:
        with open(path, "rb") as f:
            if containing.encode() not in f.read():
                continue
        text = subprocess.run([tool("llvm-objdump"), "-d", "--no-show-raw-insn", "--no-leading-addr", path], capture_output=True,
                              text=True, check=True).stdout
        for part in re.split(r"\n(?=<\S+>:)", text)[1:]:
            name = re.match(r"<(\S+)>:", part)[1]
            if containing in name:
                found[name] = re.sub(r" *//.*", "", part)  # (the encodings)
    return found


def template_numbers(symbol, kernel):
    """The template arguments (truth values and whole numbers) of `kernel` in a mangled name, or None."""
    m = re.search(rf"\d{kernel}I((?:L[bi]\d+E)+)E", symbol)
    return [int(n) for n in re.findall(r"L[bi](\d+)E", m[1])] if m else None
