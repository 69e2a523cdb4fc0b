"""GPU tests of the serving operators against their 64-bit definitions
(serving_reference.py): page plan and release, the 4-bit cache, QK norm with
rotation and its gradients, decode over the cache, and a run of them together.

Tolerances: whole numbers, cache bytes and held values are equal.  A result of
type t may be off by its rounding, half a step, and by the bound of what was
computed in fp32 before it, derived at each test (2^-24 is fp32's half step)."""
import numpy as np
import pytest
import torch

import serving_reference as R
from parity import assert_status_ok, status_word

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
I32 = torch.int32


@pytest.fixture(scope="module")
def B():
    from differential_attention_sm_b200 import binding
    binding.load()
    return binding


def np64(t):
    return t.detach().double().cpu().numpy()


def dev(a, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(a)).to(dtype).cuda() if dtype else \
        torch.as_tensor(np.ascontiguousarray(a)).cuda()


def within(got, ref, bound, what):
    g = np64(got) if isinstance(got, torch.Tensor) else got
    assert g.shape == ref.shape, (g.shape, ref.shape)
    bad = np.isnan(g) != np.isnan(ref)
    assert not bad.any(), "%s: NaN at %s" % (what, np.argwhere(bad)[:3])
    d = np.where(np.isnan(ref), 0.0, np.abs(g - ref))
    over = d > bound
    assert not over.any(), "%s: %d over, worst %.3e against %.3e" % (
        what, over.sum(), d[over].max(), np.broadcast_to(bound, d.shape)[over].min())


# ---- page plan ---------------------------------------------------------------------
def plan_state(seed, requests, page, longest, prompts, free_share, slack=0):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, longest + 1, requests)
    new = np.ones(requests, int)
    at = rng.permutation(requests)[:prompts]
    new[at] = rng.integers(0, longest + 1, prompts)
    lens[at[::2]] = 0
    new[rng.random(requests) < 0.1] = 0
    old = -(-lens // page)
    need = -(-(lens + new) // page) - old
    free = int(need.sum() * free_share)
    n_pages = int(old.sum()) + free + 3
    order = rng.permutation(n_pages)
    max_pages = max(1, -(-2 * longest // page) - slack)
    table = np.full((requests, max_pages), -1)
    p = 0
    for r in range(requests):
        for j in range(min(old[r], max_pages)):
            table[r, j] = order[p + j]
        p += old[r]
    stack = np.full(n_pages, -1)
    stack[:free] = order[old.sum():old.sum() + free]
    return new, lens, table, stack, free


@pytest.mark.parametrize("requests,page,longest,prompts,share,slots,slack", [
    (1, 16, 1, 0, 1.0, 1, 0),
    (64, 64, 3000, 0, 1.0, 64, 0),
    (33, 16, 500, 5, 0.8, 2000, 0),         # too few pages
    (70, 16, 100, 20, 1.0, 700, 0),         # too few slot rows
    (70, 32, 300, 20, 0.5, 5000, 12),       # slot rows in a launch of their own, full tables
    (1500, 16, 40, 40, 0.9, 4096, 0),       # more requests than a pass takes
    (1500, 128, 900, 30, 0.9, 20001, 1),
    (2500, 16, 7, 0, 1.0, 9000, 0),         # more requests in a CTA's rows than it keeps
    (5, 1024, 4000, 3, 1.0, 0, 0),          # no slot rows
])
def test_page_plan(B, requests, page, longest, prompts, share, slots, slack):
    new, lens, table, stack, free = plan_state(requests + page, requests, page, longest, prompts,
                                               share, slack)
    ref = R.page_plan(new, lens, table, stack, free, page, slots)
    st = status_word()
    t = dev(table, I32)
    args = (dev(new, I32), dev(lens, I32), t, dev(stack, I32), dev([free], I32), page, slots)
    got = B.diffattn_page_plan(*args, dev_status=st)
    got["block_table"] = t
    for name, want in ref.items():
        assert np.array_equal(got[name].cpu().numpy(), want), name
    assert int(st.item()) == (0 if ref["served"].all() else B.DA_ERR_CACHE_FULL)
    # again: nothing of the first call is left over
    again = B.diffattn_page_plan(*args)
    for name in again:
        assert torch.equal(again[name], got[name]), name
    # in place, as a serving loop keeps its lengths and its count
    cl, cnt = args[1].clone(), args[4].clone()
    out = dict(got, cache_lens=cl, free_count=cnt, slots=got["slots"].clone())
    B.diffattn_page_plan(args[0], cl, t, args[3], cnt, page, slots, out=out)
    assert torch.equal(cl, got["cache_lens"]) and torch.equal(cnt, got["free_count"])
    assert torch.equal(out["slots"], got["slots"])


def test_page_plan_limits(B):
    """Negative counts, a count above the pages, lengths near 2^31."""
    table = np.full((4, 2), -1)
    table[1] = [3, 1]
    new, lens = [-5, 1, 2 ** 31 - 1, 1], [-3, 31, 2 ** 31 - 1, 2 ** 31 - 1]
    stack, free = np.array([0, 2, 4, 5]), 99
    ref = R.page_plan(new, lens, table, stack, free, 16, 3)
    t = dev(table, I32)
    got = B.diffattn_page_plan(dev(new, I32), dev(lens, I32), t, dev(stack, I32), dev([free], I32),
                               16, 3)
    for name in ("slots", "served", "free_count"):
        assert np.array_equal(got[name].cpu().numpy(), ref[name]), name
    assert list(got["offsets"].cpu()) == [0, 0, 1, 2 ** 31 - 1, 2 ** 31 - 1]
    assert np.array_equal(t.cpu().numpy(), ref["block_table"])


@pytest.mark.parametrize("slots", [20, 6000])
def test_page_plan_pages_out_of_range(B, slots):
    """Entries that are no page give no slot and are reported."""
    table = np.array([[1 << 30, -1], [2, -1], [-1, -1]])
    st = status_word()
    t = dev(table, I32)
    got = B.diffattn_page_plan(dev([1, 1, 17], I32), dev([3, 3, 0], I32), t,
                               dev([0, 77, 1], I32), dev([3], I32), 16, slots, dev_status=st)
    assert list(got["slots"].cpu()[:19]) == [-1, 2 * 16 + 3] + list(range(16, 32)) + [-1]
    assert list(t.cpu()[2]) == [1, 77] and int(st.item()) == B.DA_ERR_PAGE
    assert int(got["free_count"].item()) == 1 and list(got["served"].cpu()) == [1, 1, 1]


@pytest.mark.parametrize("requests,page", [(1, 16), (37, 64), (1300, 16)])
def test_page_release(B, requests, page):
    new, lens, table, stack, free = plan_state(3, requests, page, 40 * page, 0, 1.0)
    rng = np.random.default_rng(4)
    gone = (rng.random(requests) < 0.4).astype(int)
    gone[0] = 5
    lens[0] = page + 1
    table[0, :2] = [1, 0]
    stack = np.concatenate((stack, np.full(10000, -1)))     # room for every page
    table2 = table.copy()
    want, lens2 = list(stack[:free]), lens.copy()
    for r in np.flatnonzero(gone):
        n = -(-lens[r] // page)
        want += [p for p in table[r, :n] if 0 <= p < len(stack)]
        table2[r, :n] = -1
        lens2[r] = 0
    st = status_word()
    t, s, l, c = dev(table, I32), dev(stack, I32), dev(lens, I32), dev([free], I32)
    B.diffattn_page_release(dev(gone, I32), l, t, s, c, page, dev_status=st)
    assert np.array_equal(t.cpu().numpy(), table2) and np.array_equal(l.cpu().numpy(), lens2)
    assert int(c.item()) == len(want)
    assert np.array_equal(s.cpu().numpy()[:len(want)], np.array(want))
    assert_status_ok(st)


def test_page_release_leaves_bad_entries_out(B):
    table = np.array([[3, -1, 1], [99, 2, -1], [0, -1, -1]])
    t, s = dev(table, I32), dev([5, -1, -1, -1, -1, -1], I32)
    l, c, st = dev([40, 20, 16], I32), dev([1], I32), status_word()
    B.diffattn_page_release(dev([1, 1, 0], I32), l, t, s, c, 16, dev_status=st)
    assert list(s.cpu())[:4] == [5, 3, 1, 2] and int(c.item()) == 4
    assert list(l.cpu()) == [0, 0, 16] and int(st.item()) == B.DA_ERR_PAGE


# ---- the 4-bit cache -----------------------------------------------------------------
def rows_for_cache(rng, T, H, dtype):
    x = rng.standard_normal((T, H, 128)) * np.exp(rng.standard_normal((T, H, 1)))
    flat = x.reshape(-1, 8, 16)
    if T * H > 3:
        flat[0, 0] = np.array([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5] * 2) * ([1] * 8 + [-1] * 8)
        flat[0, 1] = 0
        flat[0, 2] *= 2.0 ** -16          # subnormal scales
        flat[0, 3] *= 2.0 ** -40          # below the smallest
        flat[0, 4] *= 1e30                # saturates
        flat[1, 0, 5] = np.nan
        flat[1, 1, 2] = np.inf
        flat[1, 2, 2] = -np.inf
        flat[2, 5] = 6 * (1 + 1 / 16)     # amax / 6 between two scales
        flat[2, 6] = 6 * (1 + 3 / 16)
    return torch.tensor(x, dtype=dtype)


@pytest.mark.parametrize("T,H,page,dtype,fused", [
    (1, 1, 16, torch.bfloat16, False),
    (37, 2, 16, torch.bfloat16, True),
    (65, 8, 64, torch.float32, True),
    (130, 3, 128, torch.float32, False),
    (40, 5, 1024, torch.bfloat16, True),
])
def test_append_and_read(B, T, H, page, dtype, fused):
    rng = np.random.default_rng(T)
    k, v = rows_for_cache(rng, T, H, dtype), rows_for_cache(rng, T, H, dtype)
    if fused:   # slices of one projection [T, (4 + 1 + 1) * H * 128]
        x = torch.cat((torch.zeros(T, 4 * H * 128, dtype=dtype), k.flatten(1), v.flatten(1)), 1)
        _, kd, vd = x.cuda().split([4 * H * 128, H * 128, H * 128], 1)
        kd, vd = kd.unflatten(1, (H, 128)), vd.unflatten(1, (H, 128))
    else:
        kd, vd = k.cuda(), v.cuda()
    pages = T // page + 3
    slots = rng.permutation(pages * page)[:T]
    slots[rng.random(T) < 0.1] = -1
    before = rng.integers(0, 256, (pages, H, page * 144)).astype(np.uint8)
    cache = dev(before)
    st = status_word()
    B.diffattn_kv4_append(kd, vd, dev(slots, I32), cache, dev_status=st)
    assert_status_ok(st)
    want = before.copy()
    for x, kind in ((np64(k), "k"), (np64(v), "v")):
        sb, c = R.quantise(x)
        for t in np.flatnonzero(slots >= 0):
            p, u = slots[t] // page, slots[t] % page
            tile = want[p, :, u // 16 * 2304:][:, :2304]
            for ch in range(128):
                at, at_s = R.byte_of(kind, u % 16, ch)
                if ch % 2:
                    tile[:, at] |= c[t, :, ch] << 4
                else:
                    tile[:, at] = c[t, :, ch]
                tile[:, at_s] = sb[t, :, ch // 16]
    got = cache.cpu().numpy()
    # a negative value that rounds to 0 may be held as -0: code 8 stands for 0 too
    codes = np.tile((np.arange(2304) < 2048), page // 16)
    zero = lambda x: np.where(codes, np.where(x & 15 == 8, x & 0xF0, x), x)
    zero2 = lambda x: np.where(codes, np.where(x >> 4 == 8, x & 0x0F, x), x)
    assert np.array_equal(zero2(zero(got)), zero2(zero(want)))
    for out_dtype in (torch.bfloat16, torch.float32):
        out = tuple(torch.full((T, H, 128), 7.0, dtype=out_dtype, device="cuda") for _ in "kv")
        B.diffattn_kv4_read(cache, dev(slots, I32), out=out)
        for x, o in ((k, out[0]), (v, out[1])):
            ref = R.held(np64(x))
            ref[slots < 0] = 7.0
            assert np.array_equal(np64(o), ref, equal_nan=True)


def test_cache_skips_slots_out_of_range(B):
    cache = torch.zeros(2, 1, 16 * 144, dtype=torch.uint8, device="cuda")
    x = torch.ones(3, 1, 128, device="cuda")
    slots = dev([32, 5, 2 ** 31 - 1], I32)
    st = status_word()
    B.diffattn_kv4_append(x, x, slots, cache, dev_status=st)
    assert int(st.item()) == B.DA_ERR_PAGE
    st.zero_()
    k, v = B.diffattn_kv4_read(cache, slots, dev_status=st)
    assert int(st.item()) == B.DA_ERR_PAGE
    held = R.held(np.ones((1, 128)))
    assert np.array_equal(np64(k[1]), held) and np.array_equal(np64(v[1]), held)
    assert not k[0].any() and not k[2].any()


@pytest.mark.parametrize("dtype,off", [(torch.bfloat16, 8), (torch.float32, 4),
                                       (torch.bfloat16, 16), (torch.float32, 8)])
def test_read_into_rows_on_16_bytes(B, dtype, off):
    """Outputs that start on an odd or an even multiple of 16 bytes."""
    T, H = 21, 3
    x = torch.randn(T, H, 128, device="cuda")
    cache = torch.zeros(3, H, 16 * 144, dtype=torch.uint8, device="cuda")
    slots = torch.arange(T, dtype=I32, device="cuda")
    B.diffattn_kv4_append(x, 2 * x, slots, cache)
    want = B.diffattn_kv4_read(cache, slots, dtype=dtype)
    n = T * H * 128
    flat = torch.full((2, n + 64), 7.0, dtype=dtype, device="cuda")
    got = tuple(r[off:off + n].view(T, H, 128) for r in flat)
    assert got[0].data_ptr() % 16 == 0
    B.diffattn_kv4_read(cache, slots, out=got)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (flat[:, :off] == 7).all() and (flat[:, off + n:] == 7).all()


def test_other_streams_order_what_a_call_allocates(B):
    """Calls on a stream of their own that bring no outputs and no scratch: rows
    without a slot are 0, and the results are those of the current stream."""
    T, H = 3000, 4
    x = torch.randn(T, H, 128, device="cuda")
    cache = torch.zeros(T // 16 + 1, H, 16 * 144, dtype=torch.uint8, device="cuda")
    slots = torch.arange(T, dtype=I32, device="cuda")
    slots[::3] = -1
    B.diffattn_kv4_append(x, 2 * x, slots, cache)
    want = B.diffattn_kv4_read(cache, slots)
    pos = torch.arange(T, dtype=I32, device="cuda")
    f, w = torch.rand(64, device="cuda"), torch.rand(128, device="cuda")
    grads = B.diffattn_qk_norm_rope_bwd(x, x, x, x, pos, f, q_weight=w, k_weight=w)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        junk = torch.full((T, H, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        del junk                     # its memory may be what the next call gets
        got = B.diffattn_kv4_read(cache, slots, stream=s)
        g2 = B.diffattn_qk_norm_rope_bwd(x, x, x, x, pos, f, q_weight=w, k_weight=w,
                                         stream=s.cuda_stream)
        s.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert not got[0][::3].any()
        for name in grads:
            assert torch.equal(g2[name], grads[name]), name
        torch.cuda.synchronize()


def test_cache_no_tokens(B):
    cache = torch.zeros(2, 1, 16 * 144, dtype=torch.uint8, device="cuda")
    x = torch.ones(0, 1, 128, device="cuda")
    B.diffattn_kv4_append(x, x, torch.zeros(0, dtype=I32, device="cuda"), cache)
    k, v = B.diffattn_kv4_read(cache, torch.zeros(0, dtype=I32, device="cuda"))
    assert k.shape == v.shape == (0, 1, 128) and not cache.any()


# ---- QK norm and rotation -----------------------------------------------------------
NORM_CASES = [
    # T, Hq, Hk, d, rot, interleaved, dtype, fused, weights, far
    (1, 2, 1, 64, 64, False, torch.bfloat16, False, True, 100),
    (3, 64, 8, 128, 128, False, torch.bfloat16, True, True, 32768),
    (7, 12, 2, 128, 64, True, torch.float32, True, True, 1 << 20),
    (5, 6, 6, 64, 0, False, torch.float32, False, True, 10),
    (9, 3, 1, 32, 16, True, torch.bfloat16, True, False, 5000),
    (4, 5, 0, 16, 16, False, torch.float32, False, True, 77),
    (11, 4, 2, 256, 256, False, torch.float32, False, True, 2 ** 31 - 1),
    (6, 2, 1, 96, 32, False, torch.bfloat16, True, True, 4096),      # idle lanes
    (6, 2, 1, 240, 240, True, torch.float32, True, False, 4096),
    (1300, 3, 1, 64, 64, True, torch.bfloat16, True, True, 9000),    # batches of tokens
    (700, 40, 8, 128, 128, False, torch.bfloat16, False, True, 9000),
    (2500, 2, 2, 32, 32, False, torch.float32, True, True, 9000),
]


def norm_state(T, Hq, Hk, d, rot, dtype, fused, weights, far, seed=1):
    g = torch.Generator().manual_seed(seed + T + d)
    x = (torch.randn(T, (Hq + 2 * Hk) * d, generator=g) * 2).to(dtype)
    if T > 2:
        x[1, :d] = 0                       # a row of zeros
    q, k, _ = x.split([Hq * d, Hk * d, Hk * d], 1)
    qd, kd, _ = x.cuda().split([Hq * d, Hk * d, Hk * d], 1)
    if not fused:
        qd, kd = qd.contiguous(), kd.contiguous()
    pos = torch.randint(0, far, (T,), generator=g, dtype=I32)
    pos[0] = far - 1
    f = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float()
    w = [1 + 0.3 * torch.randn(d, generator=g) if weights else None for _ in "qk"]
    return dict(q=q.unflatten(1, (Hq, d)), k=k.unflatten(1, (Hk, d)) if Hk else None,
                qd=qd.unflatten(1, (Hq, d)), kd=kd.unflatten(1, (Hk, d)) if Hk else None,
                pos=pos, f=f if rot else None, w=w, g=g)


def cu(t):
    return None if t is None else t.cuda()


@pytest.mark.parametrize("T,Hq,Hk,d,rot,interleaved,dtype,fused,weights,far", NORM_CASES)
def test_norm_rope(B, T, Hq, Hk, d, rot, interleaved, dtype, fused, weights, far):
    s = norm_state(T, Hq, Hk, d, rot, dtype, fused, weights, far)
    eps = 1e-6
    args = (cu(s["pos"]), cu(s["f"]))
    kw = dict(q_weight=cu(s["w"][0]), k_weight=cu(s["w"][1]), norm_eps=eps,
              interleaved=interleaved)
    out = B.diffattn_qk_norm_rope(s["qd"], s["kd"], *args, **kw)
    f = None if s["f"] is None else s["f"].double().numpy()
    for x, w, got, name in zip((s["q"], s["k"]), s["w"], out, "qk"):
        if x is None:
            assert got is None
            continue
        x, w = np64(x), np.ones(d) if w is None else np64(w)
        ref = R.norm_rope(x, w, eps, s["pos"].numpy(), f, interleaved)
        flat = R.norm_rope(x, w, eps, s["pos"].numpy(), None, interleaved)
        # fp32 before the rounding: the sum (at most 16 + 4 adds: 20 half steps,
        # half of them past the root), its root (4), two products (2), cosine and
        # sine (2 steps of 1: 4), product and sum of the rotation (2).
        bound = 24 * 2.0 ** -24 * R.pair_size(flat, f, interleaved) + HALF[dtype] * np.abs(ref)
        within(got, ref, bound, name)
    # in place
    q2 = s["qd"].clone(memory_format=torch.contiguous_format)
    k2 = None if s["kd"] is None else s["kd"].clone(memory_format=torch.contiguous_format)
    B.diffattn_qk_norm_rope(q2, k2, *args, **kw, out=(q2, k2))
    assert torch.equal(q2, out[0]) and (k2 is None or torch.equal(k2, out[1]))


@pytest.mark.parametrize("T,Hq,Hk,d,rot,interleaved,dtype,fused,weights,far", NORM_CASES)
def test_norm_rope_bwd(B, T, Hq, Hk, d, rot, interleaved, dtype, fused, weights, far):
    s = norm_state(T, Hq, Hk, d, rot, dtype, fused, weights, far)
    eps = 1e-3                             # the zero row's gradient stays of a usual size
    dy = [torch.randn(T, H, d, generator=s["g"]) for H in (Hq, Hk)]
    if not Hk:
        dy[1] = None
    kw = dict(q_weight=cu(s["w"][0]), k_weight=cu(s["w"][1]), norm_eps=eps,
              interleaved=interleaved)
    args = (s["qd"], s["kd"], cu(dy[0]), cu(dy[1]), cu(s["pos"]), cu(s["f"]))
    out = B.diffattn_qk_norm_rope_bwd(*args, **kw)
    again = B.diffattn_qk_norm_rope_bwd(*args, **kw)
    f = None if s["f"] is None else s["f"].double().numpy()
    u = 2.0 ** -24
    for x, w0, g, name in zip((s["q"], s["k"]), s["w"], dy, "qk"):
        if x is None:
            assert out["d" + name] is None
            continue
        x, w, g = np64(x), np.ones(d) if w0 is None else np64(w0), np64(g)
        dx, dw = R.norm_rope_bwd(x, w, eps, s["pos"].numpy(), f, interleaved, g)
        r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        # The turned gradient is off by 6 half steps of its pair's size; r by 14
        # and a sum of d products by 24 more of its terms' sizes (see above).
        gs = R.pair_size(g, f, interleaved)
        n = np.abs(x * r)
        bound = 64 * u * r * (np.abs(w) * gs + n * (n * np.abs(w) * gs).mean(-1, keepdims=True))
        within(out["d" + name], dx, bound, "d" + name)
        assert torch.equal(out["d" + name], again["d" + name])
        if w0 is None:
            assert out["d%s_weight" % name] is None
            continue
        # each term 22 half steps, then at most T * H adds in fp32, but no more
        # than 100 in a thread's chain and 10 of a CTA at these sizes
        bound = (22 + min(T * x.shape[1], 110)) * u * (gs * n).sum((0, 1))
        within(out["d%s_weight" % name], dw, bound, "d%s_weight" % name)
        assert torch.equal(out["d%s_weight" % name], again["d%s_weight" % name])


def test_norm_rope_bwd_against_differences(B):
    """The gradients agree with differences of the GPU's own forward (fp32):
    its rounding, 24 half steps of outputs of size 4 or so over a step of 2^-7
    and a sum of d of them, is below 2e-3."""
    T, Hq, Hk, d = 2, 2, 1, 64
    s = norm_state(T, Hq, Hk, d, 64, torch.float32, False, True, 1000, seed=9)
    dy = [torch.randn(T, H, d, generator=s["g"]).cuda() for H in (Hq, Hk)]
    kw = dict(k_weight=cu(s["w"][1]), norm_eps=1e-3)
    pos, f, wq = cu(s["pos"]), cu(s["f"]), cu(s["w"][0])
    out = B.diffattn_qk_norm_rope_bwd(s["qd"], s["kd"], *dy, pos, f, q_weight=wq, **kw)

    def loss(q, k, w):
        yq, yk = B.diffattn_qk_norm_rope(q, k, pos, f, q_weight=w, **kw)
        return float((yq.double() * dy[0]).sum() + (yk.double() * dy[1]).sum())

    h = 2.0 ** -7
    for i in (0, 5, 40, 63):
        e = torch.zeros(d, device="cuda")
        e[i] = h
        num = (loss(s["qd"], s["kd"], wq + e) - loss(s["qd"], s["kd"], wq - e)) / (2 * h)
        assert abs(num - float(out["dq_weight"][i])) < 2e-3
        q = s["qd"].clone()
        q[0, 1] += e
        q2 = s["qd"].clone()
        q2[0, 1] -= e
        num = (loss(q, s["kd"], wq) - loss(q2, s["kd"], wq)) / (2 * h)
        # differences of third order: h^2 / 6 times a third derivative below 10
        assert abs(num - float(out["dq"][0, 1, i])) < 2e-3


def test_norm_rope_no_tokens_and_nan_rows(B):
    w = torch.ones(64, device="cuda")
    x = torch.zeros(0, 2, 64, device="cuda")
    e = torch.zeros(0, dtype=I32, device="cuda")
    f = torch.ones(32, device="cuda")
    q, k = B.diffattn_qk_norm_rope(x, x, e, f, q_weight=w)
    assert q.shape == (0, 2, 64)
    r = B.diffattn_qk_norm_rope_bwd(x, x, x, x, e, f, q_weight=w, k_weight=w)
    assert not r["dq_weight"].any() and not r["dk_weight"].any()
    # a NaN stays in its row; norm_eps = 0 does not leak into other rows' sums
    x = torch.randn(5, 3, 64, device="cuda")
    x[2, 1, 7] = float("nan")
    pos = torch.arange(5, dtype=I32, device="cuda")
    q, _ = B.diffattn_qk_norm_rope(x, None, pos, f, norm_eps=0.0)
    bad = torch.isnan(q).any(-1)
    assert bad[2, 1] and int(bad.sum()) == 1
    x[2, 1, 7] = 1.0
    r = B.diffattn_qk_norm_rope_bwd(x, x[:, :1].contiguous(), x, x[:, :1].contiguous(), pos, f,
                                    q_weight=w, k_weight=w, norm_eps=0.0)
    for t in r.values():
        assert torch.isfinite(t).all()


# ---- decode over the cache ------------------------------------------------------------
def decode_state(Bn, lens, Hkv, page, cols, seed=1, spare=2, extra_pages=0, bad_tail=True):
    rng = np.random.default_rng(seed)
    per = max(1, max(-(-n // page) for n in lens)) + extra_pages
    pages = sum(-(-n // page) for n in lens) + spare
    order = rng.permutation(pages)
    table = np.full((Bn, per), -1)
    p = 0
    cache = rng.integers(0, 256, (pages, Hkv, page * 144)).astype(np.uint8)
    tiles = cache.reshape(pages, Hkv, -1, 2304)
    # scales near 1 (bytes 14 .. 16 exponents), so that rows are of a usual size
    tiles[..., 2048:] = rng.integers(13 * 8, 15 * 8, tiles[..., 2048:].shape)
    for b, n in enumerate(lens):
        for j in range(-(-n // page)):
            table[b, j] = order[p]
            p += 1
        if bad_tail and n % page:    # behind the end: NaN blocks
            last = tiles[table[b, n // page]]
            for t in range(n % page, page):
                for kind in "kv":
                    for ch in range(0, 128, 16):
                        last[:, t // 16, R.byte_of(kind, t % 16, ch)[1]] = 0xFF
    q = torch.tensor(rng.standard_normal((Bn, cols, 128)), dtype=torch.bfloat16)
    return cache, table, q, rng


def check_decode(B, cache, table, lens, q, lam, form, window=0, norm=None, page=16, st_want=0,
                 **kw):
    st = status_word()
    args = (q.cuda(), dev(cache), dev(table, I32), dev(lens, I32), dev(lam, torch.float32))
    if form == 2:
        out = B.diffattn_v2_decode_kv4(*args, window=window, dev_status=st, **kw)
    else:
        opt = {} if norm is None else dict(apply_norm=True, norm_eps=norm[0],
                                           norm_weight=dev(norm[1], torch.float32),
                                           lambda_init=norm[2])
        out = B.diffattn_v1_decode_kv4(*args, window=window, dev_status=st, **opt, **kw)
    assert int(st.item()) == st_want
    Ks, Vs = (R.cache_rows(cache, table, lens, kind) for kind in "kv")
    lam32 = np.asarray(lam, np.float32).astype(np.float64)
    n64 = None if norm is None else (norm[0], np.asarray(norm[1], np.float32).astype(np.float64),
                                     1.0 - norm[2])
    for b in range(len(lens)):
        ref, bound = R.decode(np64(q[b]), Ks[b], Vs[b], lam32, form, window, n64)
        within(out[b], ref, bound + 2.0 ** -8 * np.abs(ref), "sequence %d" % b)
    return out


@pytest.mark.parametrize("lens,Hkv,group,page,window", [
    ([1], 1, 2, 16, 0),
    ([0, 1, 15, 16, 17, 31, 32, 33, 64, 65], 2, 2, 16, 0),
    ([500, 0, 1000, 3], 2, 8, 16, 0),
    ([777, 64, 128], 3, 4, 32, 0),
    ([130, 4000, 2], 2, 6, 64, 0),
    ([1025, 0, 100], 1, 10, 128, 0),            # two column tiles
    ([300, 77], 2, 16, 32, 0),
    ([300, 77, 5], 1, 34, 16, 0),               # three passes over the cache
    ([1500, 1024], 1, 8, 1024, 0),
    ([500, 10, 0, 1000, 33], 2, 8, 16, 1),      # windows
    ([500, 10, 0, 1000, 33], 2, 4, 32, 33),
    ([500, 96, 2000], 2, 12, 64, 100),
    ([0, 0], 2, 4, 16, 0),
])
def test_v2_decode(B, lens, Hkv, group, page, window):
    cache, table, q, rng = decode_state(len(lens), lens, Hkv, page, Hkv * group,
                                        seed=sum(lens) + group, extra_pages=window % 3)
    lam = rng.uniform(-0.5, 1.2, Hkv * group // 2)
    check_decode(B, cache, table, lens, q, lam, 2, window)


@pytest.mark.parametrize("lens,H,page,window,norm", [
    ([1], 1, 16, 0, True),
    ([0, 33, 500, 1], 3, 16, 0, True),
    ([700, 31], 4, 64, 0, False),
    ([700, 31, 0, 2000], 2, 128, 257, True),
])
def test_v1_decode(B, lens, H, page, window, norm):
    cache, table, q, rng = decode_state(len(lens), lens, H, page, H, seed=sum(lens))
    lam = rng.uniform(-0.5, 1.2, H)
    check_decode(B, cache, table, lens, q, lam, 1, window,
                 (1e-5, 1 + 0.2 * rng.standard_normal(128), 0.7) if norm else None)


@pytest.mark.parametrize("Bn,longest", [(700, 70), (256, 300), (257, 300)])
def test_decode_many_short_sequences(B, Bn, longest):
    """Runs that cross many sequences; both ways to find a unit's segments."""
    rng = np.random.default_rng(8)
    lens = list(rng.integers(0, longest, Bn))
    cache, table, q, rng = decode_state(Bn, lens, 2, 16, 4, seed=3)
    check_decode(B, cache, table, lens, q, rng.uniform(0, 1, 2), 2)


@pytest.mark.parametrize("q_scale", [1e-30, 1e-6, 30.0, 3e4])
def test_decode_query_sizes(B, q_scale):
    """Queries far outside fp16's range, and scores that grow along the cache."""
    lens = [900]
    cache, table, q, rng = decode_state(1, lens, 1, 16, 4, seed=12)
    tiles = cache.reshape(len(cache), 1, -1, 2304)
    for j in range(57):                       # scales rise with the position
        tiles[table[0, j], 0, 0, 2048:2176] = 8 * (8 + j // 9) + rng.integers(0, 8, 128)
    q = (q.float() * q_scale).to(torch.bfloat16)
    q[0, 1, 5] *= 2.0 ** 12
    check_decode(B, cache, table, lens, q, [0.5, 0.25], 2)


def test_decode_nan_block_and_pages_out_of_range(B):
    lens = [200, 64]
    cache, table, q, rng = decode_state(2, lens, 1, 16, 2, seed=21)
    # a NaN block of V inside a sequence: its 16 channels, nothing else
    tiles = cache.reshape(len(cache), 1, -1, 2304)
    tiles[table[0, 3], 0, 0, R.byte_of("v", 5, 32)[1]] = 0xFF
    out = check_decode(B, cache, table, lens, q, [0.4], 2)
    nan = torch.isnan(out).cpu().numpy()
    assert nan[0, 0, 32:48].all() and nan.sum() == 16
    # pages out of range are reported and their tokens take no part
    bad = table.copy()
    bad[1, 1], bad[1, 3] = len(cache), -1
    st = status_word()
    got = B.diffattn_v2_decode_kv4(q.cuda(), dev(cache), dev(bad, I32), dev(lens, I32),
                                   dev([0.4], torch.float32), dev_status=st)
    assert int(st.item()) == B.DA_ERR_PAGE
    keep = np.r_[0:16, 32:48]
    K, V = (R.cache_rows(cache, table, lens, kind)[1][:, keep] for kind in "kv")
    ref, bound = R.decode(np64(q[1]), K, V, np.array([np.float32(0.4)], np.float64), 2)
    within(got[1], ref, bound + 2.0 ** -8 * np.abs(ref), "without bad pages")


def test_decode_masked_places_hold_anything(B):
    """NaN blocks before the window's first token, in its tile and its stage;
    queries of zeros, whose weights are even."""
    lens, window = [200, 77], 60
    cache, table, q, rng = decode_state(2, lens, 1, 16, 4, seed=23)
    clean = cache.copy()
    tiles = cache.reshape(len(cache), 1, -1, 2304)
    for b, n in enumerate(lens):
        for t in range(n - window):
            for kind in "kv":
                for ch in range(0, 128, 16):
                    tiles[table[b, t // 16], 0, 0, R.byte_of(kind, t % 16, ch)[1]] = 0xFF
    q[0, 2] = 0
    q[1, 1] = 0
    out = check_decode(B, cache, table, lens, q, [0.4, -0.3], 2, window)
    assert torch.equal(out, check_decode(B, clean, table, lens, q, [0.4, -0.3], 2, window))


def test_cache_beyond_32_bits(B):
    """Pages whose bytes lie past 2^32: appended, read and attended to there as
    in a small cache."""
    pages, H, ps, n = 150000, 16, 16, 70
    cache = torch.empty(pages, H, ps * 144, dtype=torch.uint8, device="cuda")
    assert cache.numel() > 5 * 2 ** 30
    small = torch.zeros(5, H, ps * 144, dtype=torch.uint8, device="cuda")
    at = torch.tensor([pages - 1, 3, pages - 77, 120000, pages // 2], dtype=I32, device="cuda")
    near = torch.arange(5, dtype=I32, device="cuda")
    pos = torch.arange(n, device="cuda")
    slots = [(t[pos // ps] * ps + pos % ps).to(I32) for t in (at, near)]
    k, v = (torch.randn(n, H, 128, device="cuda").to(torch.bfloat16) for _ in "kv")
    for c, sl in zip((cache, small), slots):
        B.diffattn_kv4_append(k, v, sl, c)
    assert torch.equal(cache[at.long(), :, :64 * 16], small[:, :, :64 * 16])
    got, want = B.diffattn_kv4_read(cache, slots[0]), B.diffattn_kv4_read(small, slots[1])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    q = torch.randn(1, 4 * H, 128, device="cuda").to(torch.bfloat16)
    lam = torch.rand(2 * H, device="cuda")
    ln = torch.tensor([n], dtype=I32, device="cuda")
    a = B.diffattn_v2_decode_kv4(q, cache, at[None].contiguous(), ln, lam)
    b = B.diffattn_v2_decode_kv4(q, small, near[None].contiguous(), ln, lam)
    assert torch.equal(a, b) and torch.isfinite(a).all()


def test_decode_lengths_are_clamped(B):
    lens = [64, 32]
    cache, table, q, rng = decode_state(2, lens, 1, 16, 2, seed=22)
    table[1] = table[0]
    args = (q.cuda(), dev(cache), dev(table, I32))
    lam = dev([0.4], torch.float32)
    a = B.diffattn_v2_decode_kv4(*args, dev([64, -5], I32), lam)
    b = B.diffattn_v2_decode_kv4(*args, dev([2 ** 31 - 1, 0], I32), lam)
    assert torch.equal(a, b) and not a[1].any()


def test_decode_repeats_and_streams(B):
    """Equal bits from equal calls, from a captured and replayed one, and from
    calls that overlap on two streams with a workspace each."""
    lens = [3000, 1, 0, 517, 2049]
    cache, table, q, rng = decode_state(5, lens, 2, 32, 16, seed=30)
    lam = dev(rng.uniform(0, 1, 8), torch.float32)
    ln = dev(lens, I32)
    args = (q.cuda(), dev(cache), dev(table, I32), ln, lam)
    want = B.diffattn_v2_decode_kv4(*args)
    assert torch.equal(want, B.diffattn_v2_decode_kv4(*args))
    need = B.diffattn_v2_decode_kv4_workspace_size(5, 16, 2)
    ws = [torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.empty_like(want) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for w, o, s in zip(ws, outs, streams):
            B.diffattn_v2_decode_kv4(*args, workspace=w, out=o, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.diffattn_v2_decode_kv4(*args, workspace=ws[0], out=outs[0])
    outs[0].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want)
    ln.copy_(dev([100, 2, 40, 0, 7], I32))     # a replay takes the new lengths
    graph.replay()
    torch.cuda.synchronize()
    # as bits: sequence 1 now ends on a row of NaN blocks, which equals itself in no other way
    assert torch.equal(outs[0].view(torch.int16),
                       B.diffattn_v2_decode_kv4(*args).view(torch.int16))


# ---- a serving loop --------------------------------------------------------------------
def test_serving_steps(B):
    """Prompt step, decode steps with a refused request, release, and a new
    request on the freed pages: plan, norm with rotation, append, decode, as a
    server chains them on the device, against dense attention over the rows
    that the definition holds."""
    rng = np.random.default_rng(77)
    Rn, Hq, Hkv, page, n_pages, max_pages = 4, 8, 2, 16, 14, 8
    table = torch.full((Rn, max_pages), -1, dtype=I32, device="cuda")
    lens = torch.zeros(Rn, dtype=I32, device="cuda")
    stack = torch.arange(n_pages, dtype=I32, device="cuda")
    count = dev([n_pages], I32)
    cache = torch.full((n_pages, Hkv, page * 144), 0xFF, dtype=torch.uint8, device="cuda")
    lam_h = np.float32(rng.uniform(0, 1, Hq // 2))
    lam, wk = dev(lam_h), dev(np.float32(1 + 0.2 * rng.standard_normal(128)))
    f = (10000.0 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128)).float().cuda()
    kept = [[] for _ in range(Rn)]     # rows (k, v) each sequence should hold
    ref = dict(lens=np.zeros(Rn, int), table=table.cpu().numpy(), stack=stack.cpu().numpy(),
               count=n_pages)
    for step, new in enumerate([[70, 5, 0, 33], [1, 1, 1, 1], [1, 1, 0, 20], [1, 1, 90, 1],
                                "release", [0, 16, 60, 1]]):
        if new == "release":
            gone = dev([1, 0, 0, 0], I32)
            B.diffattn_page_release(gone, lens, table, stack, count, page)
            n = -(-ref["lens"][0] // page)
            ref["stack"][ref["count"]:ref["count"] + n] = ref["table"][0, :n]
            ref["count"] += n
            ref["table"][0, :n] = -1
            ref["lens"][0] = 0
            kept[0] = []
            continue
        T = sum(new) + 3
        plan = B.diffattn_page_plan(dev(new, I32), lens, table, stack, count, page, T)
        want = R.page_plan(new, ref["lens"], ref["table"], ref["stack"], ref["count"], page, T)
        for name in plan:
            assert np.array_equal(plan[name].cpu().numpy(), want[name]), (step, name)
        ref.update(lens=want["cache_lens"], table=want["block_table"],
                   count=int(want["free_count"][0]))
        lens, count = plan["cache_lens"], plan["free_count"]
        x = torch.tensor(rng.standard_normal((T, (Hq + 2 * Hkv) * 128)), dtype=torch.bfloat16)
        qd, kd, vd = x.cuda().split([Hq * 128, Hkv * 128, Hkv * 128], 1)
        qd, kd, vd = (t.unflatten(1, (-1, 128)) for t in (qd, kd, vd))
        qn, kn = B.diffattn_qk_norm_rope(qd, kd, plan["positions"], f, k_weight=wk)
        st = status_word()
        B.diffattn_kv4_append(kn, vd, plan["slots"], cache, dev_status=st)
        last = (plan["offsets"][1:] - 1).clamp(min=0).long()
        q = qn[last].contiguous()
        out = B.diffattn_v2_decode_kv4(q, cache, table, lens, lam, dev_status=st)
        assert_status_ok(st)
        hk, hv = R.held(np64(kn)), R.held(np64(vd))
        for r in range(Rn):
            if want["served"][r]:
                for i in range(want["offsets"][r], want["offsets"][r + 1]):
                    kept[r].append((hk[i], hv[i]))
            assert len(kept[r]) == ref["lens"][r]
            if kept[r]:
                K = np.stack([k for k, _ in kept[r]], 1)
                V = np.stack([v for _, v in kept[r]], 1)
            else:
                K = V = np.zeros((Hkv, 0, 128))
            o, bound = R.decode(np64(q[r]), K, V, lam_h.astype(np.float64), 2)
            within(out[r], o, bound + 2.0 ** -8 * np.abs(o), "step %d request %d" % (step, r))


def test_step_as_a_graph(B):
    """A whole step captured once and replayed with other lengths, against the
    same calls made one by one."""
    Rn, H, page, n_pages, T = 3, 2, 16, 40, 24
    i32 = dict(dtype=I32, device="cuda")

    def state():
        return dict(new=torch.ones(Rn, **i32), lens=torch.zeros(Rn, **i32),
                    table=torch.full((Rn, 10), -1, **i32), stack=torch.arange(n_pages, **i32),
                    count=torch.full((1,), n_pages, **i32),
                    cache=torch.zeros(n_pages, H, page * 144, dtype=torch.uint8, device="cuda"))

    g = torch.Generator().manual_seed(3)
    x = torch.randn(T, 8 * 128, generator=g).to(torch.bfloat16).cuda()
    f = (10000.0 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128)).float().cuda()
    w, lam = torch.ones(128, device="cuda"), torch.tensor([0.2, 0.7], device="cuda")
    ws = torch.empty(B.diffattn_v2_decode_kv4_workspace_size(Rn, 4, H), dtype=torch.uint8,
                     device="cuda")

    def step(s):
        q, k, v = (t.unflatten(1, (-1, 128)) for t in x.split([512, 256, 256], 1))
        p = B.diffattn_page_plan(s["new"], s["lens"], s["table"], s["stack"], s["count"], page, T)
        q, k = B.diffattn_qk_norm_rope(q, k, p["positions"], f, q_weight=w, k_weight=w)
        B.diffattn_kv4_append(k, v, p["slots"], s["cache"])
        last = (p["offsets"][1:] - 1).clamp(min=0).long()
        out = B.diffattn_v2_decode_kv4(q[last], s["cache"], s["table"], p["cache_lens"], lam,
                                       workspace=ws)
        s["lens"].copy_(p["cache_lens"])
        s["count"].copy_(p["free_count"])
        return out

    a, b = state(), state()
    step(b)                       # warm-up, on a state that is then put back
    fresh = state()
    for name in b:
        b[name].copy_(fresh[name])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(b)
    for new in ([5, 17, 1], [1, 1, 1], [1, 0, 16], [2, 9, 1]):
        for s in (a, b):
            s["new"].copy_(torch.tensor(new, dtype=I32))
        want = step(a)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        for name in a:
            assert torch.equal(a[name], b[name]), name


def test_norm_backward_as_a_graph(B):
    s = norm_state(300, 6, 2, 128, 128, torch.bfloat16, True, True, 5000)
    dy = [torch.randn(300, H, 128, generator=s["g"]).cuda() for H in (6, 2)]
    args = (s["qd"], s["kd"], *dy, cu(s["pos"]), cu(s["f"]))
    kw = dict(q_weight=cu(s["w"][0]), k_weight=cu(s["w"][1]))
    want = B.diffattn_qk_norm_rope_bwd(*args, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = B.diffattn_qk_norm_rope_bwd(*args, **kw)
    for t in got.values():
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for name in want:
        assert torch.equal(got[name], want[name]), name
    # in place, as the attention's gradients are of no further use
    q = dy[0].clone()
    lib = B.load()
    ws = torch.empty(B.diffattn_qk_norm_rope_bwd_workspace_size(300, 6, 2, 128),
                     dtype=torch.uint8, device="cuda")
    k = dy[1].clone()
    st = lib.diffattn_qk_norm_rope_bwd(
        s["qd"].data_ptr(), s["qd"].stride(0), s["kd"].data_ptr(), s["kd"].stride(0), B.DA_BF16,
        q.data_ptr(), 6 * 128, k.data_ptr(), 2 * 128, 300, 6, 2, 128,
        kw["q_weight"].data_ptr(), kw["k_weight"].data_ptr(), 1e-6, args[4].data_ptr(),
        args[5].data_ptr(), 128, 0, q.data_ptr(), k.data_ptr(), None, None, ws.data_ptr(),
        ws.nbytes, torch.cuda.current_stream().cuda_stream)
    assert st == B.DA_OK and torch.equal(q, want["dq"]) and torch.equal(k, want["dk"])


def test_norm_gradient_continues_the_attention_backward(B):
    """Training path: norm with rotation, V2 prefill, its backward, and the
    norm's backward from the attention's fp32 gradients, in place."""
    T, Hq, Hkv, d = 96, 4, 2, 128
    s = norm_state(T, Hq, Hkv, d, 128, torch.bfloat16, True, True, T, seed=4)
    pos = torch.arange(T, dtype=I32, device="cuda")
    kw = dict(q_weight=cu(s["w"][0]), k_weight=cu(s["w"][1]), norm_eps=1e-6)
    q, k = B.diffattn_qk_norm_rope(s["qd"], s["kd"], pos, cu(s["f"]), **kw)
    v = torch.randn(1, T, Hkv, d, generator=s["g"]).to(torch.bfloat16).cuda()
    lam = torch.tensor([0.3, 0.6], device="cuda")
    do = torch.randn(1, T, Hq // 2, d, generator=s["g"]).to(torch.bfloat16).cuda()
    g = B.diffattn_v2_bwd(q[None], k[None], v, do, lam)
    r = B.diffattn_qk_norm_rope_bwd(s["qd"], s["kd"], g["dq"][0], g["dk"][0], pos, cu(s["f"]),
                                    **kw)
    f = s["f"].double().numpy()
    for name, x, w in (("q", s["q"], s["w"][0]), ("k", s["k"], s["w"][1])):
        dx, dw = R.norm_rope_bwd(np64(x), np64(w), 1e-6, pos.cpu().numpy(), f, False,
                                 np64(g["d" + name][0]))
        scale = np.abs(dx).max()
        # rows of zeros aside (their r is 1000), 2^-16 of the largest is far above 64 half steps
        live = np.abs(np64(x)).sum(-1) > 0
        assert np.abs(np64(r["d" + name]) - dx)[live].max() <= 2.0 ** -16 * scale
        assert np.isfinite(np64(r["d%s_weight" % name])).all()
