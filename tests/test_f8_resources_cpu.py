"""Registers of the built kernels of the F8 products and codec, dropout and the embedding, from the
code objects' own metadata, without a GPU: none may spill to scratch memory."""
import os
import struct

import pytest

from test_mx_resources_cpu import BUNDLE, notes


@pytest.fixture(scope="module")
def kernels():
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
    return found


@pytest.mark.parametrize("family", ["k_f8_gemm", "k_f8_split", "k_f8_few", "k_f8_rows", "k_f8_quantize", "k_f8_dequantize", "k_dropout",
                                    "k_embedding_sort", "k_embedding_sums", "k_embedding_join", "k_embedding_count",
                                    "k_embedding_scan", "k_embedding_move", "11k_embedding", "k_mx_embedding"])
def test_no_scratch(kernels, family):
    own = {n: k for n, k in kernels.items() if family in n}
    assert own
    spilled = {n: k[".private_segment_fixed_size"] for n, k in own.items()
               if k[".private_segment_fixed_size"] or k[".vgpr_spill_count"]}
    assert not spilled
