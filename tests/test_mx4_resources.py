"""What the built kernels of the 4-bit products and the experts' layer ask of a
compute unit, read from the metadata that the compiler writes for each."""

import struct

import pytest

import sparse_dense_matmul_amd as sdm

msgpack = pytest.importorskip("msgpack")

DEFAULT_LDS = 64 * 1024  # more has to be allowed for a kernel first
TILES = ("6k_tileI", "11k_tile_gradI", "11k_tile_bothI", "8k_streamI", "13k_stream_gradI", "13k_stream_bothI")
# bytes of LDS that a launch adds at most: the sums of 128 tokens, staged tokens
DYNAMIC = {"k_experts_down": 8 * 128 * 64, "k_experts_up_few": 48 * 1024}


def device_images(data):
    """The gfx950 ELF images of the library's offload bundles."""
    at = data.find(b"__CLANG_OFFLOAD_BUNDLE__")
    while at >= 0:
        (count,), p = struct.unpack_from("<Q", data, at + 24), at + 32
        for _ in range(count):
            offset, size, name = struct.unpack_from("<QQQ", data, p)
            target = data[p + 24:p + 24 + name]
            p += 24 + name
            if b"gfx950" in target and size:
                yield data[at + offset:at + offset + size]
        at = data.find(b"__CLANG_OFFLOAD_BUNDLE__", at + 24)


def kernels(elf):
    """The entries of the image's AMDGPU metadata note."""
    shoff, = struct.unpack_from("<Q", elf, 0x28)
    entry, count = struct.unpack_from("<HH", elf, 0x3A)
    for i in range(count):
        kind, = struct.unpack_from("<I", elf, shoff + i * entry + 4)
        offset, size = struct.unpack_from("<QQ", elf, shoff + i * entry + 0x18)
        p, end = offset, offset + size
        while kind == 7 and p < end:  # SHT_NOTE
            name, desc, note = struct.unpack_from("<III", elf, p)
            body = p + 12 + (name + 3) // 4 * 4
            if note == 32 and elf[p + 12:p + 12 + name].startswith(b"AMDGPU"):
                yield from msgpack.unpackb(elf[body:body + desc])["amdhsa.kernels"]
            p = body + (desc + 3) // 4 * 4


@pytest.fixture(scope="module")
def built():
    with open(sdm.LIB_PATH, "rb") as fh:
        data = fh.read()
    all_of = [k for image in device_images(data) for k in kernels(image)]
    mine = [k for k in all_of if any(n in k[".name"] for n in ("k_experts", "k_few", "quantize") + TILES)]
    assert len(mine) > 60
    return mine


def test_no_kernel_spills(built):
    for k in built:
        assert k[".private_segment_fixed_size"] == 0, k[".name"]


def test_shared_memory_stays_within_what_is_allowed(built):
    for name, dynamic in DYNAMIC.items():
        found = [k for k in built if name in k[".name"]]
        assert found
        for k in found:
            assert k[".group_segment_fixed_size"] + dynamic <= DEFAULT_LDS, k[".name"]
    # those allowed as much as they ask for have no more than 1 KB besides
    for name in TILES:
        found = [k for k in built if name in k[".name"]]
        assert found and all(k[".group_segment_fixed_size"] <= 1024 for k in found), name
