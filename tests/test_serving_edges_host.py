"""Host side of the serving operators at their edges: the decode's index rules,
compiled from the kernel's own header by the host compiler, and calls that are
refused.  No device."""
import ctypes
import os
import subprocess

import pytest
import torch

import readme_step
import serving_reference as R

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "differential_attention_sm_b200", "csrc")
A = 0x10000   # 16-byte aligned fake device address
NO_TILE, BAD_TILE = 0xFFFFFFFF, 0xFFFFFFFE


@pytest.fixture(scope="module")
def b():
    from differential_attention_sm_b200 import build
    build.build()
    from differential_attention_sm_b200 import binding
    binding.load()
    return binding


@pytest.fixture(scope="module")
def index(tmp_path_factory):
    d = tmp_path_factory.mktemp("index")
    src = d / "index.cpp"
    src.write_text('#include "kv4_index.h"\n'
                   'extern "C" int joined(unsigned a, unsigned b) '
                   '{ return da::tiles_joined(a, b); }\n'
                   'extern "C" void span(int* v, int runs) '
                   '{ da::bound_span(v[0], v[1], runs); }\n')
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


def test_spans_of_a_unit_stay_within_the_scratch(index):
    """Spans that no warp wrote (its wait timed out) hold anything.  The scratch
    has a slot for each unit and one for each run: slot unit + first + i, with
    i below count, is inside it."""
    edge = [-2 ** 31, -2 ** 31 + 1, -1, 0, 1, 2, 1183, 1184, 1185, 1775, 1776, 1777, 2 ** 30,
            2 ** 31 - 2, 2 ** 31 - 1]
    for runs in (1184, 1776):
        for first in edge:
            for count in edge:
                v = (ctypes.c_int * 2)(first, count)
                index.span(v, runs)
                assert v[0] >= 0 and v[1] >= 0 and v[0] + v[1] <= runs, (first, count, list(v))
                if 0 <= first and 0 <= count and first + count <= runs:
                    assert list(v) == [first, count]


def test_v1_decode_refuses_an_odd_width(b):
    """Half of it would pass for a branch, and the rows for rows of 128."""
    i32 = dict(dtype=torch.int32)
    cache = torch.zeros(3, 4, 16 * 144, dtype=torch.uint8)
    for width in (127, 129):
        q = torch.zeros(5, 4, width, dtype=torch.bfloat16)
        with pytest.raises(ValueError, match="width"):
            b.diffattn_v1_decode_kv4(q, cache, torch.zeros(5, 2, **i32), torch.zeros(5, **i32),
                                     torch.zeros(4))


def test_page_plan_refuses_a_workspace_between_words(b):
    """Its kernels keep int32 there; a slice of a byte buffer may begin anywhere."""
    ws = b.diffattn_page_plan_workspace_size(4, 273)
    for off in (1, 2, 3):
        args = [A] * 5 + [4, 8, 100, 64, 273] + [A] * 6 + [A + off, ws, None, None]
        assert b.load().diffattn_page_plan(*args) == b.DA_ERR_ALIGNMENT


def test_marshalling_module_of_another_torch_is_refused(b, monkeypatch):
    """It is compiled against one torch's C++ interface."""
    monkeypatch.setattr(b, "_marshal", None)
    with monkeypatch.context() as other:
        other.setattr(torch, "__version__", "0.0.0")
        with pytest.raises(ImportError, match="0.0.0"):
            b._serving()
    assert b._marshal is None and b._serving().torch_version == torch.__version__


# ---- the step that the documents show ----------------------------------------------
class Definitions:
    """The calls of a serving step by their definitions, on the CPU."""

    @staticmethod
    def diffattn_page_plan(new, lens, table, stack, count, page, n_slots):
        r = R.page_plan(new.numpy(), lens.numpy(), table.numpy(), stack.numpy(), int(count), page,
                        n_slots)
        table.copy_(torch.as_tensor(r.pop("block_table")))
        return {k: torch.as_tensor(v).to(torch.int32) for k, v in r.items()}

    @staticmethod
    def diffattn_qk_norm_rope(q, k, positions, inv_freq, *, q_weight, k_weight):
        assert len(positions) == len(q)
        return q, k

    @staticmethod
    def diffattn_kv4_append(k, v, slots, cache):
        assert len(slots) == len(k)

    @staticmethod
    def diffattn_v2_decode_kv4(q, cache, table, lens, lam):
        return torch.zeros(q.shape[0], q.shape[1] // 2, 128)

    @staticmethod
    def diffattn_page_release(release, lens, table, stack, count, page):
        for r in range(len(release)):
            for j in range(-(-int(lens[r]) // page) if release[r] else 0):
                stack[int(count)] = table[r, j]
                table[r, j] = -1
                count += 1
            if release[r]:
                lens[r] = 0


def test_readme_step_keeps_the_page_pool():
    readme_step.run(Definitions, "cpu")
