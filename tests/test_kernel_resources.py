"""Registers and LDS of the built kernels, from the metadata in the library:
what the plans' workgroups per compute unit rest on (host only)."""
import struct

import pytest

import permute_grouped_gemm_amd as pgg

msgpack = pytest.importorskip("msgpack")
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"
CU_LDS = 160 * 1024


def _code_objects(blob):
    """The gfx950 ELF images of every offload bundle in the library."""
    at = blob.find(MAGIC)
    while at >= 0:
        n, = struct.unpack_from("<Q", blob, at + len(MAGIC))
        p = at + len(MAGIC) + 8
        for _ in range(n):
            off, size, length = struct.unpack_from("<QQQ", blob, p)
            triple = blob[p + 24:p + 24 + length]
            p += 24 + length
            if triple.endswith(b"gfx950") and size:
                yield blob[at + off:at + off + size]
        at = blob.find(MAGIC, at + 1)


def _kernels(elf):
    """The kernels' metadata: the AMDGPU note of an ELF64 image."""
    shoff, = struct.unpack_from("<Q", elf, 0x28)
    shentsize, shnum = struct.unpack_from("<HH", elf, 0x3A)
    for i in range(shnum):
        kind, = struct.unpack_from("<I", elf, shoff + i * shentsize + 4)
        if kind != 7:   # SHT_NOTE
            continue
        off, size = struct.unpack_from("<QQ", elf, shoff + i * shentsize + 0x18)
        namesz, descsz, note = struct.unpack_from("<III", elf, off)
        if note == 32:
            desc = off + 12 + (namesz + 3) // 4 * 4
            yield from msgpack.unpackb(elf[desc:desc + descsz], strict_map_key=False)["amdhsa.kernels"]


@pytest.fixture(scope="module")
def kernels():
    pgg.lib()
    with open(pgg.LIB_PATH, "rb") as f:
        blob = f.read()
    found = {k[".name"]: k for elf in _code_objects(blob) for k in _kernels(elf)}
    assert len(found) > 50
    return found


def test_no_kernel_spills_vector_registers(kernels):
    assert not [n for n, k in kernels.items() if k[".vgpr_spill_count"]]


# rows of the tile -> workgroups per compute unit that the gradient's plan splits for
@pytest.mark.parametrize("rows,resident", [(32, 4), (64, 3), (128, 2)])
def test_the_gradients_workgroups_fit_a_compute_unit(kernels, rows, resident):
    mine = [k for n, k in kernels.items() if "glu_grad_reg_kernel" in n and f"Li{rows}ELi128E" in n]
    assert len(mine) == 6   # 3 types, 2 activations
    for k in mine:
        assert k[".group_segment_fixed_size"] * resident <= CU_LDS
        # 4 waves to a workgroup, one to each SIMD of 512 registers
        assert k[".vgpr_count"] * resident <= 512


@pytest.mark.parametrize("name,resident", [("few_kernelINS", 2), ("pipe_kernelINS", 1), ("nn_reg_kernelINS", 2)])
def test_the_tiles_workgroups_fit_a_compute_unit(kernels, name, resident):
    mine = [k for n, k in kernels.items() if name in n]
    assert mine
    for k in mine:
        assert k[".group_segment_fixed_size"] * resident <= CU_LDS
        waves = k[".max_flat_workgroup_size"] // 256   # to a SIMD
        assert (k[".vgpr_count"] + 7) // 8 * 8 * resident * waves <= 512
