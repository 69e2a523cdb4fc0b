"""Host side of the serving operators (page plan, QK norm with rotation, 4-bit
cache, decode over it): arguments are refused before anything is enqueued, and
the 64-bit definitions the GPU tests use agree with each other.  No device."""
import numpy as np
import pytest
import torch

import serving_reference as R

A = 0x10000   # 16-byte aligned fake device address
U = 0x10008   # misaligned


@pytest.fixture(scope="module")
def b():
    from differential_attention_sm_b200 import build
    build.build()
    from differential_attention_sm_b200 import binding
    binding.load()
    return binding


def refuses(f, ok, changes):
    for at, value, status in changes:
        bad = list(ok)
        for i, v in zip(at if isinstance(at, tuple) else (at,),
                        value if isinstance(at, tuple) else (value,)):
            bad[i] = v
        assert f(*bad) == status, (at, value)


def test_status_strings(b):
    assert b.status_string(b.DA_ERR_PAGE) == "DA_ERR_PAGE"
    assert b.status_string(b.DA_ERR_CACHE_FULL) == "DA_ERR_CACHE_FULL"


def test_page_plan_refusals(b):
    inv, uns = b.DA_ERR_INVALID_ARG, b.DA_ERR_UNSUPPORTED
    assert b.diffattn_page_plan_workspace_size(4, 272) == 0
    ws = b.diffattn_page_plan_workspace_size(4, 273)
    assert ws > 0
    ok = [A] * 5 + [4, 8, 100, 64, 7] + [A] * 6 + [None, 0, None, None]
    refuses(b.load().diffattn_page_plan, ok, [
        *((i, None, inv) for i in (0, 1, 2, 3, 4, 10, 11, 12, 13, 14, 15)),
        (5, 0, inv), (6, 0, inv), (7, 0, inv), (8, 0, inv), (9, -1, inv),
        (8, 48, uns), (8, 8, uns), (8, 2048, uns), (5, (1 << 16) + 1, uns),
        (7, 1 << 25, uns), (6, 1 << 25, uns), (9, (1 << 30) + 1, uns),
        (9, 273, b.DA_ERR_WORKSPACE), ((9, 16, 17), (273, A, ws - 1), b.DA_ERR_WORKSPACE)])
    ok = [A] * 5 + [4, 8, 100, 64, None, None]
    refuses(b.load().diffattn_page_release, ok, [
        *((i, None, inv) for i in range(5)), (5, 0, inv), (8, 24, uns)])


def test_cache_refusals(b):
    inv, uns, ali = b.DA_ERR_INVALID_ARG, b.DA_ERR_UNSUPPORTED, b.DA_ERR_ALIGNMENT
    assert b.diffattn_kv4_page_bytes(8, 128, 64) == 8 * 64 * 144
    for bad in ((0, 128, 64), (8, 64, 64), (8, 128, 8), (8, 128, 100), (8, 128, 0)):
        assert b.diffattn_kv4_page_bytes(*bad) == 0
    ok = [A, 1024, A, 1024, b.DA_BF16, A, 5, 8, 128, A, 10, 64, None, None]
    refuses(b.load().diffattn_kv4_append, ok, [
        *((i, None, inv) for i in (0, 2, 5, 9)), (4, 9, inv), (6, -1, inv), (7, 0, inv),
        (1, 1023, inv), (3, 512, inv), (10, 0, inv), (8, 64, uns), (11, 100, uns),
        (10, 1 << 25, uns), (6, (1 << 31) - 1, uns), (1, 1028, ali), (3, 1025, ali), (0, U, ali),
        (2, U, ali), (9, U, ali)])
    assert b.load().diffattn_kv4_append(*[*ok[:6], 0, *ok[7:]]) == b.DA_OK   # no tokens
    ok = [A, 10, 64, A, 5, 8, 128, A, A, b.DA_BF16, None, None]
    refuses(b.load().diffattn_kv4_read, ok, [
        *((i, None, inv) for i in (0, 3, 7, 8)), (9, 5, inv), (6, 64, uns), (2, 4096, uns),
        (0, U, ali), (7, U, ali), (8, U, ali)])
    assert b.load().diffattn_kv4_read(*[*ok[:4], 0, *ok[5:]]) == b.DA_OK


def test_decode_refusals(b):
    inv, uns, ali, ws_ = (b.DA_ERR_INVALID_ARG, b.DA_ERR_UNSUPPORTED, b.DA_ERR_ALIGNMENT,
                          b.DA_ERR_WORKSPACE)
    ws = b.diffattn_v2_decode_kv4_workspace_size(4, 64, 8)
    assert ws > 0 and ws % 16 == 0
    for bad in ((0, 64, 8), (4, 64, 7), (4, 24, 8), (4, 64, 0), (1 << 21, 64, 8)):
        assert b.diffattn_v2_decode_kv4_workspace_size(*bad) == 0
    ok = [A, A, 100, 64, A, 8, A, 0, A, b.DA_BF16, 4, 64, 8, 128, A, A, ws, None, None]
    refuses(b.load().diffattn_v2_decode_kv4, ok, [
        *((i, None, inv) for i in (0, 1, 4, 6, 8, 14)), (7, -1, inv), (9, 3, inv), (10, 0, inv),
        (11, 63, inv), (11, 24, inv), (12, 0, inv), (2, 0, inv), (5, 0, inv),
        (9, b.DA_FP32, uns), (13, 64, uns), (3, 40, uns), (10, 1 << 21, uns), (2, 1 << 25, uns),
        (0, U, ali), (1, U, ali), (8, U, ali), (15, U, ali), (15, None, ws_), (16, ws - 1, ws_)])
    ws = b.diffattn_v1_decode_kv4_workspace_size(4, 16)
    assert ws > 0 and b.diffattn_v1_decode_kv4_workspace_size(4, 0) == 0
    ok = [A, A, 100, 64, A, 8, A, 0, A, b.DA_BF16, 4, 16, 64, 128, A, 1, None, 1e-5, 0.2, A, ws,
          None, None]
    refuses(b.load().diffattn_v1_decode_kv4, ok, [
        *((i, None, inv) for i in (0, 1, 4, 6, 8, 14)), (17, -1.0, inv), (17, float("nan"), inv),
        (12, 32, uns), (13, 64, uns), (9, b.DA_FP32, uns), (0, U, ali), (19, None, ws_),
        (20, ws - 1, ws_), (19, U, ali)])


def test_norm_rope_refusals(b):
    inv, uns, ali = b.DA_ERR_INVALID_ARG, b.DA_ERR_UNSUPPORTED, b.DA_ERR_ALIGNMENT
    ok = [A, 2048, A, 512, b.DA_BF16, 7, 16, 4, 128, A, A, 1e-6, A, A, 128, 0, A, 2048, A, 512,
          None]
    refuses(b.load().diffattn_qk_norm_rope, ok, [
        *((i, None, inv) for i in (0, 2, 12, 13, 16, 18)), (4, 2, inv), (5, -1, inv), (6, 0, inv),
        (7, -1, inv), (11, -1.0, inv), (14, 144, inv), (14, -16, inv), (1, 2040, inv),
        (17, 2040, inv), (3, 504, inv),
        ((8, 14), (100, 96), uns), ((8, 1, 3, 17, 19), (272, 8192, 8192, 8192, 8192), uns),
        (14, 24, uns), (1, 2052, ali), (19, 516, ali), (0, U, ali), (2, U, ali), (9, U, ali),
        (10, U, ali), (16, U, ali), (18, U, ali)])
    assert b.load().diffattn_qk_norm_rope(*[*ok[:5], 0, *ok[6:]]) == b.DA_OK
    ws = b.diffattn_qk_norm_rope_bwd_workspace_size(7, 16, 4, 128)
    assert ws > 0 and b.diffattn_qk_norm_rope_bwd_workspace_size(7, 16, 4, 100) == 0
    ok = [A, 2048, A, 512, b.DA_FP32, A, 2048, A, 512, 7, 16, 4, 128, A, A, 1e-6, A, A, 64, 1, A,
          A, A, A, A, ws, None]
    refuses(b.load().diffattn_qk_norm_rope_bwd, ok, [
        *((i, None, inv) for i in (0, 2, 5, 7, 20, 21)), (6, 1024, inv), (8, 514, ali),
        (5, U, ali), (7, U, ali), (20, U, ali), (21, U, ali), (24, U, ali),
        (24, None, b.DA_ERR_WORKSPACE), (25, ws - 1, b.DA_ERR_WORKSPACE)])


def test_binding_refuses_host_tensors_and_wrong_shapes(b):
    i32 = dict(dtype=torch.int32)
    cache = torch.zeros(3, 2, 16 * 144, dtype=torch.uint8)
    rows = torch.zeros(5, 2, 128, dtype=torch.bfloat16)
    slots = torch.zeros(5, **i32)
    with pytest.raises(ValueError, match="CUDA"):
        b.diffattn_kv4_append(rows, rows, slots, cache)
    with pytest.raises(TypeError, match="slots"):
        b.diffattn_kv4_append(rows, rows, slots.long(), cache)
    with pytest.raises(ValueError, match="slots"):
        b.diffattn_kv4_append(rows, rows, slots[:4], cache)
    with pytest.raises(ValueError, match="cache"):
        b.diffattn_kv4_append(rows[:, :1], rows[:, :1], slots, cache)
    with pytest.raises(ValueError, match="in a row"):
        b.diffattn_kv4_append(rows.transpose(0, 1).contiguous().transpose(0, 1), rows, slots,
                              cache)
    with pytest.raises(TypeError, match="v must be"):
        b.diffattn_kv4_append(rows, rows.float(), slots, cache)
    with pytest.raises(TypeError, match="dev_status"):
        b.diffattn_kv4_append(rows, rows, slots, cache, dev_status=slots.to(torch.uint8))
    with pytest.raises(TypeError, match="k must be a tensor"):
        b.diffattn_kv4_append(None, rows, slots, cache)
    with pytest.raises(TypeError, match="dtype"):
        b.diffattn_kv4_read(cache, slots, dtype=torch.float16)
    with pytest.raises(ValueError, match="out of range"):
        b.diffattn_page_plan(slots, slots, torch.zeros(5, 2, **i32), slots, slots[:1], 16, 1 << 40)
    with pytest.raises(ValueError, match="page_size"):
        b.diffattn_kv4_read(torch.zeros(3, 2, 100, dtype=torch.uint8), slots)
    q = torch.zeros(5, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="block_table"):
        b.diffattn_v2_decode_kv4(q, cache, torch.zeros(4, 2, **i32), slots, torch.zeros(2))
    with pytest.raises(TypeError, match="cache_lens"):
        b.diffattn_v2_decode_kv4(q, cache, torch.zeros(5, 2, **i32), slots.long(), torch.zeros(2))
    with pytest.raises(ValueError, match="lam"):
        b.diffattn_v2_decode_kv4(q, cache, torch.zeros(5, 2, **i32), slots, torch.zeros(4))
    with pytest.raises(ValueError, match="cache"):
        b.diffattn_v1_decode_kv4(q, cache, torch.zeros(5, 2, **i32), slots, torch.zeros(4))
    with pytest.raises(ValueError, match="positions"):
        b.diffattn_qk_norm_rope(rows, rows, slots[:3], torch.zeros(64))
    with pytest.raises(TypeError, match="inv_freq"):
        b.diffattn_qk_norm_rope(rows, rows, slots, torch.zeros(64, dtype=torch.float64))
    with pytest.raises(ValueError, match="width"):
        b.diffattn_qk_norm_rope(rows, rows[..., :64].contiguous(), slots, torch.zeros(32))
    with pytest.raises(ValueError, match="shapes"):
        b.diffattn_qk_norm_rope_bwd(rows, rows, rows.float()[:, :1], rows.float(), slots, None)
    with pytest.raises(ValueError, match="served"):
        b.diffattn_page_plan(slots, slots, torch.zeros(5, 2, **i32), slots, slots[:1], 16, 5,
                             out=dict(slots=slots, positions=slots,
                                      offsets=torch.zeros(6, **i32), served=slots[:2],
                                      cache_lens=slots, free_count=slots[:1]))


# ---- the definitions themselves -------------------------------------------------
def test_tile_bytes_are_a_partition():
    used = np.zeros(2304, int)
    for kind in "kv":
        for t in range(16):
            for c in range(0, 128, 2):
                at, at_s = R.byte_of(kind, t, c)
                assert at == R.byte_of(kind, t, c + 1)[0]
                used[at] += 1
                used[at_s] += 1
    assert (used[:2048] == 1).all() and (used[2048:] == 8).all()


def test_quantiser_ties_and_limits():
    x = np.zeros((6, 128))
    x[0, :16] = [6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, -6]
    x[1, :16] = 1e6                       # saturates
    x[2, 3] = np.nan
    x[3, 3] = -np.inf
    x[4, :16] = 2.0 ** -30                # below the smallest scale
    x[5, :2] = [6 * (1 + 1 / 16), 1]      # amax / 6 halfway between two scales: even
    sb, c = R.quantise(x)
    assert sb[0, 0] == 15 * 8 and sb[1, 0] == 0xE2 and sb[2, 0] == sb[3, 0] == 0xFF
    assert sb[4, 0] == 0 and sb[5, 0] == 15 * 8
    assert list(c[0, :16]) == [7, 0, 2, 2, 4, 4, 6, 6, 0, 10, 10, 12, 12, 14, 14, 15]
    h = R.held(x)
    assert (h[1, :16] == 61440).all() and np.isnan(h[2, :16]).all() and (h[2, 16:] == 0).all()
    assert (h[4] == 0).all()


def test_norm_rope_gradient_against_differences():
    rng = np.random.default_rng(5)
    for interleaved in (False, True):
        x, dy = rng.standard_normal((2, 3, 32)), rng.standard_normal((2, 3, 32))
        w, pos = 1 + 0.3 * rng.standard_normal(32), np.array([3, 70000])
        f = np.array([1.0, 0.3, 0.05, 0.01, 0.4, 0.002, 0.7, 0.9])
        loss = lambda x_, w_: (R.norm_rope(x_, w_, 1e-3, pos, f, interleaved) * dy).sum()
        dx, dw = R.norm_rope_bwd(x, w, 1e-3, pos, f, interleaved, dy)
        for at in ((0, 0, 0), (1, 2, 9), (0, 1, 17), (1, 0, 31)):
            h = np.zeros_like(x)
            h[at] = 1e-5
            assert abs((loss(x + h, w) - loss(x - h, w)) / 2e-5 - dx[at]) < 1e-7
        for i in (0, 5, 20):
            h = np.zeros(32)
            h[i] = 1e-5
            assert abs((loss(x, w + h) - loss(x, w - h)) / 2e-5 - dw[i]) < 1e-7


def test_plan_definition():
    table = np.full((3, 4), -1)
    table[0, :2] = [7, 3]
    r = R.page_plan([1, 5, 1], [32, 0, 0], table, np.array([9, 8, 5, -1]), 3, 16, 8)
    assert list(r["slots"]) == [5 * 16, 8 * 16, 8 * 16 + 1, 8 * 16 + 2, 8 * 16 + 3, 8 * 16 + 4,
                                9 * 16, -1]
    assert list(r["positions"]) == [32, 0, 1, 2, 3, 4, 0, 0] and r["free_count"] == [0]
