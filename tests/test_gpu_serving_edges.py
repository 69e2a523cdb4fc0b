"""GPU tests of the serving operators at their edges, against the same 64-bit
definitions (serving_reference.py) and with the same tolerances as
test_gpu_serving.py."""
import numpy as np
import pytest
import torch

import readme_step
import serving_reference as R
import test_gpu_serving as S
from parity import status_word
from test_gpu_serving import check_decode, decode_state, dev, np64, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from differential_attention_sm_b200 import binding
    binding.load()
    return binding


# ---- page plan: what a server keeps --------------------------------------------------
def test_kept_lengths_do_not_hold_the_slot_map(B):
    """The lengths and the count that the next step takes lie apart from a large
    step's slot map."""
    R_, n = 5, 50000
    i32 = dict(dtype=torch.int32, device="cuda")
    table, stack = torch.full((R_, 800), -1, **i32), torch.arange(4000, **i32)
    args = (torch.full((R_,), 9000, **i32), torch.zeros(R_, **i32), table, stack,
            torch.full((1,), 4000, **i32), 16, n)
    plan = B.diffattn_page_plan(*args)
    for name in ("cache_lens", "free_count"):
        assert plan[name].untyped_storage().nbytes() <= 4 * (R_ + 1)
    ref = R.page_plan([9000] * R_, [0] * R_, np.full((R_, 800), -1), np.arange(4000), 4000, 16, n)
    for name in plan:
        assert np.array_equal(plan[name].cpu().numpy(), ref[name]), name


# ---- decode: windows that begin inside a stage ---------------------------------
@pytest.mark.parametrize("form", [1, 2])
@pytest.mark.parametrize("tile", [0, 1, 2, 3, 5, 7, 9, 33])
def test_window_before_the_first_tile_of_the_cache(B, form, tile):
    """One head and pages of one tile, taken in order from page 0 behind a
    window's first tile: what stands for the tiles before it is no neighbour of
    the cache's first tile."""
    n_tiles = tile + 9
    lens = [16 * n_tiles - 5]
    window = lens[0] - 16 * tile - 3
    cache, table, q, rng = decode_state(1, lens, 1, 16, form, seed=tile, spare=0,
                                        bad_tail=False)
    table[0, :n_tiles] = [n_tiles - tile + j for j in range(tile)] + list(range(n_tiles - tile))
    assert sorted(table[0, :n_tiles]) == list(range(n_tiles))
    check_decode(B, cache, table, lens, q, [0.4], form, window)


# ---- decode: nothing to attend to, and queries that are no numbers ----------------
@pytest.mark.parametrize("eps", [0.0, 1e-5])
def test_v1_norm_of_a_sequence_without_visible_tokens(B, eps):
    """All of its pages out of range: 0, also where the norm has no epsilon."""
    lens = [40, 17, 0]
    cache, table, q, rng = decode_state(3, lens, 2, 16, 2, seed=31, bad_tail=False)
    table[1] = [len(cache), -1, 1 << 30]
    st = status_word()
    out = B.diffattn_v1_decode_kv4(q.cuda(), dev(cache), dev(table, torch.int32),
                                   dev(lens, torch.int32), dev([0.4, 0.3], torch.float32),
                                   apply_norm=True, norm_eps=eps, dev_status=st)
    assert int(st.item()) == B.DA_ERR_PAGE
    assert not out[1].any() and not out[2].any() and out[0].any() and torch.isfinite(out).all()


@pytest.mark.parametrize("form", [1, 2])
@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
def test_queries_that_are_no_numbers(B, form, value):
    """Scores of infinities have no softmax: NaN wherever there is a token, also
    if every score is the lowest; 0 where there is none; other heads as ever."""
    lens, H = [40, 0, 130], 2
    cache = torch.zeros(16, H, 16 * 144, dtype=torch.uint8, device="cuda")
    ones = torch.ones(16 * 16, H, 128, device="cuda")          # every score has q's sign
    g = torch.Generator().manual_seed(8)
    v = torch.randn(16 * 16, H, 128, generator=g).cuda()
    B.diffattn_kv4_append(ones, v, torch.arange(256, dtype=torch.int32, device="cuda"), cache)
    table = torch.arange(3 * 9, dtype=torch.int32, device="cuda").remainder(16).view(3, 9)
    q = torch.randn(3, H * form * 2 if form == 2 else H, 128, generator=g).to(torch.bfloat16)
    ln = dev(lens, torch.int32)
    run = B.diffattn_v1_decode_kv4 if form == 1 else B.diffattn_v2_decode_kv4
    lam = torch.rand(H if form == 1 else H * 2, generator=g).cuda()
    clean = run(q.cuda(), cache, table, ln, lam)
    for b in range(3):
        q[b, 1, 70] = value              # V1: branch 2 of head 1; V2: pair 0's second head
    out = run(q.cuda(), cache, table, ln, lam)
    hit = 1 if form == 1 else 0
    for b in (0, 2):
        assert torch.isnan(out[b, hit]).all()
    out[:, hit] = clean[:, hit]
    assert torch.equal(out, clean) and torch.isfinite(clean).all()
    assert not clean[1].any()
    if value != value:
        return
    only = torch.full_like(q, float(value)).cuda()
    full = run(only, cache, table, ln, lam)
    assert torch.isnan(full[0]).all() and torch.isnan(full[2]).all() and not full[1].any()


# ---- norm: infinities -----------------------------------------------------------------
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 0), (64, 32), (128, 128), (96, 16), (256, 128)])
def test_norm_of_an_infinity(B, d, rot, interleaved, dtype):
    """1 / sqrt(mean) is 0 there: the infinity's own place is NaN, and its
    partner's if it is rotated; every other feature is 0."""
    g = torch.Generator().manual_seed(d + rot)
    x = torch.randn(6, 3, d, generator=g).to(dtype)
    for t, (at, v) in enumerate([(0, np.inf), (d - 1, -np.inf), (d // 2 + 3, np.inf),
                                 (min(rot, d - 1), np.inf), (max(rot - 1, 0), np.inf)]):
        x[t, 1, at] = v
    pos = torch.tensor([0, 1, 5, 0, 70000, 2], dtype=torch.int32)
    f = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float()
    w = 1 + 0.3 * torch.randn(d, generator=g)
    got, _ = B.diffattn_qk_norm_rope(x.cuda(), None, pos.cuda(), f.cuda() if rot else None,
                                     q_weight=w.cuda(), interleaved=interleaved)
    f64 = f.double().numpy() if rot else None
    args = (np64(x), np64(w), 1e-6, pos.numpy())
    with np.errstate(invalid="ignore"):
        ref = R.norm_rope(*args, f64, interleaved)
        size = R.pair_size(R.norm_rope(*args, None, interleaved), f64, interleaved)
    bound = 24 * 2.0 ** -24 * size + (2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -24) * \
        np.abs(ref)
    within(got, ref, np.where(np.isnan(bound), 0, bound), "q")


# ---- norm: gradients of the weights ------------------------------------------------
def test_weight_gradient_of_many_rows(B):
    """Sums of rows that all round the same way: 1023 of a thread, each 1 + 0.45
    * 2^-14, which a running fp32 sum above 512 cuts to 1.  The bound counts 22
    half steps of a term, 128 of the adds that are in fp32 and 6 behind them,
    however many rows there are; a chain of them all is off by 205."""
    H, d = 32, 256
    T = 1023 * 148 * 2 * 16 // H           # two CTAs an SM, 16 rows of a CTA at a time
    x = torch.ones(T, H, d, dtype=torch.bfloat16, device="cuda")
    c = float(np.float32(1 + 0.45 * 2.0 ** -14))
    dy = torch.full((T, H, d), c, device="cuda")
    w = torch.ones(d, device="cuda")
    got = B.diffattn_qk_norm_rope_bwd(x, None, dy, None, None, None, q_weight=w, norm_eps=0.0)
    want = T * H * c
    worst = float((got["dq_weight"].double() - want).abs().max())
    assert worst <= (22 + 128 + 6) * 2.0 ** -24 * want, worst / want * 2.0 ** 24
    # all of the gradient lies along x: w dy - x mean(x w dy) is 0 but for the
    # rounding of a sum of 256 and of the root
    assert float(got["dq"].abs().max()) <= 64 * 2.0 ** -24 * c


# ---- the step that the documents show ----------------------------------------------
def test_readme_step_keeps_the_page_pool(B):
    readme_step.run(B, "cuda")


# ---- main loops: more work than the grid has places ---------------------------------
def long_state(lens, Hkv, page, cols, seed, pages=24):
    """A few distinct pages, used over and over; scores that rise and fall from
    page to page by more than the running maximum's slack."""
    rng = np.random.default_rng(seed)
    cache = rng.integers(0, 256, (pages, Hkv, page * 144)).astype(np.uint8)
    tiles = cache.reshape(pages, Hkv, -1, 2304)
    tiles[..., 2048:] = rng.integers(13 * 8, 15 * 8, tiles[..., 2048:].shape)
    tiles[..., 2048:2176] += (8 * (np.arange(pages) % 4)).astype(np.uint8)[:, None, None, None]
    per = max(1, -(-max(lens) // page))
    table = rng.integers(0, pages, (len(lens), per))
    table[::3] = (table[::3, :1] + np.arange(per)) % pages     # neighbours in memory, too
    for b, n in enumerate(lens):
        table[b, -(-n // page):] = -1
    q = torch.tensor(rng.standard_normal((len(lens), cols, 128)), dtype=torch.bfloat16)
    rows = [np.stack(R.cache_rows(cache, np.arange(pages)[:, None], [page] * pages, kind))
            for kind in "kv"]                                  # [pages][heads, page, 128]
    return cache, table, q, rng, rows


@pytest.mark.parametrize("form,Bn,longest,Hkv,group,page,window", [
    (2, 200, 3600, 3, 2, 64, 0),            # one column tile; segments found by sums
    (2, 330, 3000, 2, 8, 16, 0),            # segments written down
    (2, 1, 72001, 16, 2, 32, 0),            # one sequence over all warps
    (2, 400, 4100, 2, 4, 16, 1500),
    (2, 340, 4300, 1, 10, 32, 0),           # two column tiles
    (2, 1, 45000, 16, 12, 64, 0),
    (1, 150, 3600, 5, 1, 64, 0),
    (1, 300, 3000, 3, 1, 16, 2200),
])
def test_decode_of_many_stages(B, form, Bn, longest, Hkv, group, page, window):
    """Runs of 10 stages and more, which pass from head to head and from sequence
    to sequence: each warp's ring goes round, its tile indices are looked up anew,
    and its maximum and sums are carried from stage to stage."""
    rng = np.random.default_rng(Bn + Hkv)
    lens = [longest] if Bn == 1 else list(rng.integers(longest // 2, longest, Bn))
    if Bn > 1:
        lens[5], lens[6], lens[90] = 0, 1, 64
    lens = [int(n) for n in lens]
    cache, table, q, rng, (Kp, Vp) = long_state(lens, Hkv, page, Hkv * group, seed=Bn + page)
    chunks = -(-group // 16)
    seen = [(max(0, n - window) if window else 0, n) for n in lens]
    stages = sum((n - 1) // 64 - lo // 64 + 1 for lo, n in seen if n) * Hkv * chunks
    warps = 148 * (12 if group <= 8 else 8)
    assert stages > 9 * warps, stages
    lam = rng.uniform(-0.5, 1.2, Hkv if form == 1 else Hkv * group // 2)
    st = status_word()
    run = B.diffattn_v1_decode_kv4 if form == 1 else B.diffattn_v2_decode_kv4
    args = (q.cuda(), dev(cache), dev(table, torch.int32), dev(lens, torch.int32),
            dev(lam, torch.float32))
    out = run(*args, window=window, dev_status=st)
    assert int(st.item()) == 0
    assert torch.equal(out, run(*args, window=window))
    lam64 = np.asarray(lam, np.float32).astype(np.float64)
    some = range(Bn) if Bn == 1 else sorted({5, 6, 90, *rng.permutation(Bn)[:60].tolist()})
    heads = group // 2 if form == 2 else 1          # outputs of a KV head
    q64 = np64(q)
    for b in some:
        n = lens[b]
        for h in range(Hkv):
            at = table[b, :-(-n // page)]
            K, V = (x[at, h].reshape(-1, 128)[None, :n] for x in (Kp, Vp))
            sl = slice(h * heads, (h + 1) * heads)
            ref, bound = R.decode(q64[b, h * group:(h + 1) * group], K, V, lam64[sl], form, window)
            within(out[b, sl], ref, bound + 2.0 ** -8 * np.abs(ref), "sequence %d head %d" % (b, h))


@pytest.mark.parametrize("case", [
    # T, Hq, Hk, d, rot, interleaved, dtype, fused, weights, far
    (3000, 32, 8, 128, 128, False, torch.bfloat16, True, True, 1 << 20),
    (3000, 32, 8, 128, 64, True, torch.float32, False, True, 9000),
    (9001, 5, 2, 64, 64, True, torch.bfloat16, True, True, 9000),
    (6000, 3, 1, 256, 128, False, torch.float32, True, False, 9000),
    (20000, 2, 0, 32, 32, False, torch.float32, False, True, 30000),
])
def test_norm_of_many_batches(B, case):
    """CTAs that take several batches of tokens: both angle buffers, and rows on
    their way from one batch into the next; forward and backward."""
    S.test_norm_rope(B, *case)
    S.test_norm_rope_bwd(B, *case)


@pytest.mark.parametrize("T,H,page,dtype", [
    (8000, 16, 64, torch.bfloat16),
    (8000, 16, 16, torch.float32),
    (30000, 3, 32, torch.bfloat16),
    (30000, 7, 128, torch.float32),
])
def test_append_and_read_of_many_rows(B, T, H, page, dtype):
    """CTAs that walk over the heads: the next row on its way while one is packed,
    and several heads' codes asked for at once; byte by byte."""
    rng = np.random.default_rng(T + H)
    base = S.rows_for_cache(rng, 300, 1, dtype)[:, 0]             # rows, used over and over
    idx = [rng.integers(0, 300, (T, H)) for _ in "kv"]
    kd, vd = (base[torch.as_tensor(i)].cuda() for i in idx)
    pages = T // page + 3
    slots = rng.permutation(pages * page)[:T]
    slots[rng.random(T) < 0.05] = -1
    before = rng.integers(0, 256, (pages, H, page * 144)).astype(np.uint8)
    cache, st = dev(before), status_word()
    B.diffattn_kv4_append(kd, vd, dev(slots, torch.int32), cache, dev_status=st)
    assert int(st.item()) == 0
    want = before.copy()
    sb, codes = R.quantise(np64(base))
    live = np.flatnonzero(slots >= 0)
    p, u = slots[live] // page, slots[live] % page
    head = np.arange(H)[None, :, None]
    for kind, i in zip("kv", idx):
        at, at_s = R.byte_of(kind, np.arange(16)[:, None], np.arange(0, 128, 2)[None])
        where = (u // 16 * 2304)[:, None] + at[u % 16]
        pair = codes[:, 0::2] | (codes[:, 1::2] << 4)
        want[p[:, None, None], head, where[:, None]] = pair[i[live]]
        _, at_s = R.byte_of(kind, np.arange(16)[:, None], np.arange(0, 128, 16)[None])
        where = (u // 16 * 2304)[:, None] + at_s[u % 16]
        want[p[:, None, None], head, where[:, None]] = sb[i[live]]
    got = cache.cpu().numpy()
    # a negative value that rounds to 0 may be held as -0: code 8 stands for 0 too
    is_code = np.tile(np.arange(2304) < 2048, page // 16)
    for x in (got, want):
        c = x[..., is_code]
        c = np.where(c & 15 == 8, c & 0xF0, c)
        x[..., is_code] = np.where(c >> 4 == 8, c & 0x0F, c)
    assert np.array_equal(got, want)
    held = R.held(np64(base))
    for out_dtype in (torch.bfloat16, torch.float32):
        out = tuple(torch.full((T, H, 128), 7.0, dtype=out_dtype, device="cuda") for _ in "kv")
        B.diffattn_kv4_read(cache, dev(slots, torch.int32), out=out)
        for i, o in zip(idx, out):
            ref = held[i]
            ref[slots < 0] = 7.0
            assert np.array_equal(np64(o), ref, equal_nan=True)


# ---- calls that are allowed and rare -------------------------------------------------
def test_step_captured_over_two_streams(B):
    """A step whose norm runs beside the plan and joins it before the append: each
    call's launches wait for both of what they come after."""
    Rn, H, page, n_pages, T = 300, 2, 16, 700, 900
    i32 = dict(dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(3)
    x = torch.randn(T, 8, 128, generator=g).to(torch.bfloat16).cuda()
    pos = torch.arange(T, **i32)
    f = torch.rand(64, generator=g).cuda()
    lam = torch.tensor([0.2, 0.7], device="cuda")
    ws = torch.empty(B.diffattn_v2_decode_kv4_workspace_size(Rn, 4, H), dtype=torch.uint8,
                     device="cuda")
    table, stack = torch.full((Rn, 4), -1, **i32), torch.arange(n_pages, **i32)
    new = torch.tensor([1 + i % 5 for i in range(Rn)], **i32)
    lens, count = torch.zeros(Rn, **i32), torch.full((1,), n_pages, **i32)
    cache = torch.zeros(n_pages, H, page * 144, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()

    def step(other):
        main = torch.cuda.current_stream()
        if other is not None:
            other.wait_stream(main)
        q, k = B.diffattn_qk_norm_rope(x[:, :4], x[:, 4:6], pos, f, stream=other)
        p = B.diffattn_page_plan(new, lens, table, stack, count, page, T)
        if other is not None:
            main.wait_stream(other)
        B.diffattn_kv4_append(k, x[:, 6:], p["slots"], cache)
        last = (p["offsets"][1:] - 1).long()
        return p, B.diffattn_v2_decode_kv4(q[last], cache, table, p["cache_lens"], lam,
                                           workspace=ws)

    p, want = step(None)
    want, slots = want.clone(), p["slots"].clone()
    assert bool(p["served"].all()) and torch.isfinite(want).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p, out = step(side)
    for _ in range(5):
        cache.zero_()
        table.fill_(-1)
        for t in (out, p["slots"], p["cache_lens"]):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(p["slots"], slots)


def test_norm_of_a_token_of_very_many_heads(B):
    S.test_norm_rope(B, 1, 100000, 3, 16, 16, False, torch.bfloat16, False, True, 70)
    # the weights' gradient by terms of one sign: 22 half steps of a term, 128 adds
    # in fp32 and 6 behind them
    g = torch.Generator().manual_seed(1)
    x = torch.rand(1, 100000, 16, generator=g) + 0.5
    dy = torch.rand(1, 100000, 16, generator=g) + 0.5
    w = torch.ones(16)
    got = B.diffattn_qk_norm_rope_bwd(x.cuda(), None, dy.cuda(), None, None, None,
                                      q_weight=w.cuda())
    dx, dw = R.norm_rope_bwd(np64(x), np64(w), 1e-6, np.zeros(1), None, False, np64(dy))
    within(got["dq_weight"], dw, (22 + 128 + 6) * 2.0 ** -24 * np.abs(dw), "dq_weight")


def test_positions_before_the_first(B):
    """Angles of negative positions turn the other way, to the far end of int32."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn(4, 2, 64, generator=g)
    pos = torch.tensor([-1, -2 ** 31, 2 ** 31 - 1, -4097], dtype=torch.int32)
    f = (10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).float()
    got, _ = B.diffattn_qk_norm_rope(x.cuda(), None, pos.cuda(), f.cuda())
    args = (np64(x), np.ones(64), 1e-6, pos.numpy())
    f64 = f.double().numpy()
    size = R.pair_size(R.norm_rope(*args, None, False), f64, False)
    within(got, R.norm_rope(*args, f64, False), 25 * 2.0 ** -24 * size, "q")


def test_release_and_plan_take_turns_in_a_graph(B):
    """A captured release and plan, replayed: the pages go round and none is lost."""
    Rn, page, n_pages = 40, 16, 64
    i32 = dict(dtype=torch.int32, device="cuda")
    table, stack = torch.full((Rn, 4), -1, **i32), torch.arange(n_pages, **i32)
    lens, count = torch.zeros(Rn, **i32), torch.full((1,), n_pages, **i32)
    gone, new = torch.zeros(Rn, **i32), torch.zeros(Rn, **i32)
    out = dict(slots=torch.empty(600, **i32), positions=torch.empty(600, **i32),
               offsets=torch.empty(Rn + 1, **i32), served=torch.empty(Rn, **i32),
               cache_lens=lens, free_count=count)
    ws = torch.empty(B.diffattn_page_plan_workspace_size(Rn, 600), dtype=torch.uint8,
                     device="cuda")

    def step():
        B.diffattn_page_release(gone, lens, table, stack, count, page)
        B.diffattn_page_plan(new, lens, table, stack, count, page, 600, out=out, workspace=ws)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rng = np.random.default_rng(1)
    for _ in range(12):
        gone.copy_(torch.as_tensor((rng.random(Rn) < 0.3).astype(np.int32)))
        new.copy_(torch.as_tensor(rng.integers(0, 20, Rn).astype(np.int32)))
        graph.replay()
        held = [int(t) for row, n in zip(table.tolist(), lens.tolist())
                for t in row[:-(-n // page)]]
        assert sorted(held + stack.tolist()[:int(count)]) == list(range(n_pages))


@pytest.mark.parametrize("T,Hq,Hk,d,rot,interleaved,dtype", [
    (700, 5, 3, 16, 16, False, torch.bfloat16),      # several rows of a line of memory
    (3000, 32, 8, 128, 128, True, torch.bfloat16),
    (41, 3, 2, 48, 16, False, torch.float32),
])
def test_norm_in_place_on_a_fused_projection(B, T, Hq, Hk, d, rot, interleaved, dtype):
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, (Hq + 2 * Hk) * d, generator=g).to(dtype).cuda()
    before = x.clone()
    q, k, v = (t.unflatten(1, (-1, d)) for t in x.split([Hq * d, Hk * d, Hk * d], 1))
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    f = torch.rand(rot // 2, generator=g).cuda()
    w = torch.rand(d, generator=g).cuda()
    kw = dict(q_weight=w, interleaved=interleaved)
    want = B.diffattn_qk_norm_rope(q, k, pos, f, **kw)
    assert torch.equal(x, before)
    B.diffattn_qk_norm_rope(q, k, pos, f, **kw, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(x[:, (Hq + Hk) * d:], before[:, (Hq + Hk) * d:])


def test_streams_by_number_and_by_object(B):
    """The default stream is number 0."""
    x = torch.randn(64, 3, 128, device="cuda")
    pos = torch.arange(64, dtype=torch.int32, device="cuda")
    f = torch.rand(64, device="cuda")
    want = B.diffattn_qk_norm_rope(x, None, pos, f)[0]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for s in (0, torch.cuda.default_stream(), side, side.cuda_stream, None):
        got = B.diffattn_qk_norm_rope(x, None, pos, f, stream=s)[0]
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    with torch.cuda.stream(side):
        got = B.diffattn_qk_norm_rope(x, None, pos, f)[0]
        side.synchronize()
        assert torch.equal(got, want) and torch.cuda.current_stream() == side


@pytest.mark.parametrize("T,Hq,Hk,d,rot,interleaved,dtype", [
    (12000, 96, 30, 128, 64, True, torch.bfloat16),
    (20000, 100, 30, 64, 64, False, torch.float32),
    (25001, 90, 31, 48, 16, False, torch.bfloat16),        # idle lanes
    (9000, 40, 31, 256, 256, False, torch.float32),
])
def test_norm_gradients_of_very_many_rows(B, T, Hq, Hk, d, rot, interleaved, dtype):
    """More rows of a thread than it adds up in fp32 (queries, keys, both layouts),
    against the formulas in 64 bits."""
    lanes = 1 << (max(d - 1, 0) // 16).bit_length()
    assert T * (Hq + Hk) > 128 * 296 * (256 // lanes)
    g = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    pos = torch.randint(0, 9000, (T,), generator=g, device="cuda", dtype=torch.int32)
    f = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()
    x = [rnd(T, H, d).to(dtype) for H in (Hq, Hk)]
    dy = [rnd(T, H, d) for H in (Hq, Hk)]
    w = [1 + 0.3 * rnd(d) for _ in "qk"]
    eps = 1e-3
    args = (*x, *dy, pos, f)
    kw = dict(q_weight=w[0], k_weight=w[1], norm_eps=eps, interleaved=interleaved)
    out = B.diffattn_qk_norm_rope_bwd(*args, **kw)
    again = B.diffattn_qk_norm_rope_bwd(*args, **kw)
    for name in out:
        assert torch.equal(out[name], again[name]), name
    ang = pos.double()[:, None] * f.double()
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    i = torch.arange(rot // 2, device="cuda")
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    u = 2.0 ** -24
    for xx, yy, ww, name in zip(x, dy, w, "qk"):
        xx, yy, ww = xx.double(), yy.double(), ww.double()
        t, gs = yy.clone(), yy.abs()
        t[..., a] = yy[..., a] * c + yy[..., b] * s
        t[..., b] = yy[..., b] * c - yy[..., a] * s
        gs[..., a] = gs[..., b] = yy[..., a].abs() + yy[..., b].abs()
        r = 1 / (xx.square().mean(-1, keepdim=True) + eps).sqrt()
        n, wg = xx * r, ww * t
        dx = r * (wg - n * (n * wg).mean(-1, keepdim=True))
        size = r * (ww.abs() * gs + n.abs() * (n.abs() * ww.abs() * gs).mean(-1, keepdim=True))
        assert bool(((out["d" + name].double() - dx).abs() <= 64 * u * size).all()), name
        dw, terms = (t * n).sum((0, 1)), (gs * n.abs()).sum((0, 1))
        off = (out["d%s_weight" % name].double() - dw).abs()
        assert bool((off <= (22 + 128 + 6) * u * terms).all()), name
