"""Host side of the serving operators at their edges: the decode's index rules,
compiled from the kernel's own header by the host compiler.  No device."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "differential_attention_sm_b200", "csrc")
NO_TILE, BAD_TILE = 0xFFFFFFFF, 0xFFFFFFFE


@pytest.fixture(scope="module")
def index(tmp_path_factory):
    d = tmp_path_factory.mktemp("index")
    src = d / "index.cpp"
    src.write_text('#include "kv4_index.h"\n'
                   'extern "C" int joined(unsigned a, unsigned b) '
                   '{ return da::tiles_joined(a, b); }\n')
    so = d / "index.so"
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I" + CSRC, str(src), "-o",
                    str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    lib.joined.argtypes = [ctypes.c_uint, ctypes.c_uint]
    return lib


def test_only_tiles_of_the_cache_are_joined(index):
    """A stage is one copy from its first tile's address if its tiles are
    neighbours; what stands for no tile has no address."""
    for mine in (0, 1, 7, 0x7FFFFFFF, BAD_TILE - 2):
        assert index.joined(mine, mine + 1)
        assert not index.joined(mine, mine) and not index.joined(mine, mine + 2)
    for none in (NO_TILE, BAD_TILE):
        for other in (0, 1, BAD_TILE - 1, BAD_TILE, NO_TILE):
            assert not index.joined(none, other), (none, other)
            assert not index.joined(other, none), (other, none)
