"""The gfx950 kernels of a built library: size, registers and instructions, read from the
code objects that hipcc bundles in it."""
import struct
import subprocess

import msgpack

MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"
OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


def code_objects(path):
    """Every gfx950 ELF of the library, one per source file."""
    data = open(path, "rb").read()
    at = data.find(MAGIC)
    while at >= 0:
        count, = struct.unpack_from("<Q", data, at + 24)
        p = at + 32
        if count > 16:                      # (the magic inside some other data)
            count = 0
        for _ in range(count):
            offset, size, idlen = struct.unpack_from("<QQQ", data, p)
            if size and b"gfx950" in data[p + 24:p + 24 + idlen]:
                yield data[at + offset:at + offset + size]
            p += 24 + idlen
        at = data.find(MAGIC, at + 24)


def kernels(elf):
    """{name: metadata} of one code object."""
    table, = struct.unpack_from("<Q", elf, 40)
    entry, count = struct.unpack_from("<HH", elf, 58)
    out = {}
    for i in range(count):
        _, kind, _, _, offset, size = struct.unpack_from("<IIQQQQ", elf, table + i * entry)
        p, end = offset, offset + size
        while kind == 7 and p < end:        # notes: name length, length, type, name, contents
            namelen, length, note = struct.unpack_from("<III", elf, p)
            at = p + 12 + (namelen + 3) // 4 * 4
            if note == 32:
                out.update((k[".name"], k) for k in msgpack.unpackb(elf[at:at + length])["amdhsa.kernels"])
            p = at + (length + 3) // 4 * 4
    return out


def instructions(path, symbols):
    """{symbol: its mnemonics} of a code object on disk."""
    text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--disassemble-symbols=" + ",".join(symbols), path],
                          check=True, capture_output=True, text=True).stdout
    out, now = {}, None
    for line in text.splitlines():
        if line.endswith(">:"):
            now = out.setdefault(line[line.index("<") + 1:-2], [])
        elif now is not None and line.startswith("\t"):
            now.append(line.split()[0])
    return out
