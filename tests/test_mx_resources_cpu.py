"""Registers of the built MX kernels, from the code objects' own metadata, without a GPU: the
products hold their sums in registers, and a lane that spills some of them to scratch memory
waits for it in every stage."""
import struct

import pytest

msgpack = pytest.importorskip("msgpack")

BUNDLE = b"__CLANG_OFFLOAD_BUNDLE__"


def notes(elf):
    """The kernels of one gfx950 code object (an ELF file): its metadata note."""
    (phoff,), (size, count) = struct.unpack_from("<Q", elf, 32), struct.unpack_from("<HH", elf, 54)
    for i in range(count):
        kind, _, at, _, _, length = struct.unpack_from("<IIQQQQ", elf, phoff + i * size)
        end = at + length
        while kind == 4 and at < end:
            name, desc, note = struct.unpack_from("<III", elf, at)
            body = at + 12 + (name + 3) // 4 * 4
            if elf[at + 12:at + 12 + name] == b"AMDGPU\0" and note == 32:
                yield from msgpack.unpackb(elf[body:body + desc], strict_map_key=False)["amdhsa.kernels"]
            at = body + (desc + 3) // 4 * 4


@pytest.fixture(scope="module")
def kernels():
    import os
    from bit_optimizers_block_amd import bitopt
    if not os.path.exists(bitopt.LIB_PATH):
        from bit_optimizers_block_amd import build
        build.build()
    with open(bitopt.LIB_PATH, "rb") as f:
        data = f.read()
    found, at = {}, data.find(BUNDLE)
    while at >= 0:
        (entries,), p = struct.unpack_from("<Q", data, at + 24), at + 32
        for _ in range(entries):
            offset, size, length = struct.unpack_from("<QQQ", data, p)
            if b"gfx950" in data[p + 24:p + 24 + length]:
                found.update((k[".name"], k) for k in notes(data[at + offset:at + offset + size]))
            p += 24 + length
        at = data.find(BUNDLE, at + 24)
    return {n: k for n, k in found.items() if "k_mx_" in n or "k_swiglu" in n}


@pytest.mark.parametrize("family", ["k_mx_gemm16", "k_mx_gemm4", "k_mx_skinny", "k_mx_tokens", "k_mx_quantize",
                                    "k_mx_dequantize", "k_swiglu_forward", "k_swiglu_backward"])
def test_no_scratch(kernels, family):
    own = {n: k for n, k in kernels.items() if family in n}
    assert own
    spilled = {n: k[".private_segment_fixed_size"] for n, k in own.items()
               if k[".private_segment_fixed_size"] or k[".vgpr_spill_count"]}
    assert not spilled
