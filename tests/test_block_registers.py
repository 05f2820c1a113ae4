"""What the compiler made of the residual block's kernels, from the metadata of
the built library (no GPU)."""
import os
import re
import struct

import pytest

LIB = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rl_experience_collection_amd",
                   "librollout.so")


@pytest.fixture(scope="module")
def kernels():
    """Kernel name: its metadata, from the AMDGPU notes of the code objects."""
    msgpack = pytest.importorskip("msgpack")
    if not os.path.exists(LIB):
        pytest.skip("the library is not built")
    raw = open(LIB, "rb").read()
    found = {}
    for m in re.finditer(rb"AMDGPU\x00\x00", raw):
        name, size, kind = struct.unpack_from("<III", raw, m.start() - 12)
        if (name, kind) != (7, 32):
            continue
        note = msgpack.unpackb(raw[m.end():m.end() + size], strict_map_key=False)
        found.update((k[".name"], k) for k in note["amdhsa.kernels"])
    assert found
    return found


def test_no_forward_norm_spills_registers(kernels):
    norms = {n: k for n, k in kernels.items() if "norm_forward_kernel" in n}
    assert norms
    assert not {n: k[".vgpr_spill_count"] for n, k in norms.items() if k[".vgpr_spill_count"]}
