"""Scratch memory of the built kernels, from the metadata that the compiler writes into
libssd.so's code objects (no GPU needed).

Registers that do not fit go to scratch, which every row of a norm or chunk of a walk
then reads and writes.  Kernels of the block operators hold at most 256 bytes per lane
there: 64 fp32 values.  (A form of the widest norms' gradients held 1656, and took fifteen
times as long.)"""
import struct

import msgpack
import pytest

import mamba_ssd_chunked_fwd_amd as ssd

BLOCK = ("walk_kernel", "run_starts_kernel", "sum_heads_kernel", "linattn_step_kernel",
         "add_norm_fwd_kernel", "add_norm_bwd_kernel", "gated_norm_fwd_kernel",
         "gated_norm_bwd_kernel", "sum_rows_kernel")


def code_objects(data):
    """The gfx950 ELF images of a shared library's offload bundles."""
    magic = b"__CLANG_OFFLOAD_BUNDLE__"
    at = data.find(magic)
    while at >= 0:
        n, = struct.unpack_from("<Q", data, at + len(magic))
        p = at + len(magic) + 8
        for _ in range(n):
            off, size, idlen = struct.unpack_from("<QQQ", data, p)
            name = data[p + 24:p + 24 + idlen]
            p += 24 + idlen
            if b"gfx950" in name and size:
                yield data[at + off:at + off + size]
        at = data.find(magic, at + 1)


def kernels(elf):
    """The kernels' entries of a code object's metadata note."""
    phoff, = struct.unpack_from("<Q", elf, 32)
    phsize, phnum = struct.unpack_from("<HH", elf, 54)
    for i in range(phnum):
        kind, = struct.unpack_from("<I", elf, phoff + i * phsize)
        off, = struct.unpack_from("<Q", elf, phoff + i * phsize + 8)
        size, = struct.unpack_from("<Q", elf, phoff + i * phsize + 32)
        if kind != 4:                          # PT_NOTE
            continue
        p = off
        while p < off + size:
            nlen, dlen, what = struct.unpack_from("<III", elf, p)
            desc = p + 12 + (nlen + 3) // 4 * 4
            if what == 32 and elf[p + 12:p + 18] == b"AMDGPU":
                yield from msgpack.unpackb(elf[desc:desc + dlen])["amdhsa.kernels"]
            p = desc + (dlen + 3) // 4 * 4


@pytest.fixture(scope="module")
def scratch():
    with open(ssd.LIB_PATH, "rb") as f:
        data = f.read()
    return {k[".name"]: k[".private_segment_fixed_size"]
            for elf in code_objects(data) for k in kernels(elf)}


@pytest.mark.parametrize("kernel", BLOCK)
def test_scratch_of_the_block_operators(scratch, kernel):
    sizes = {n: s for n, s in scratch.items() if kernel in n}
    assert sizes, "not in the library"
    worst = max(sizes, key=sizes.get)
    assert sizes[worst] <= 256, (worst, sizes[worst])
