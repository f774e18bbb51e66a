"""GPU tests of the paged key/value cache and the attention over it against plain 64-bit forms."""
import numpy as np
import pytest
import torch

import megatron_tensor_transformer_colwise_gb300 as tp
import oracle
import synth
from gpu_util import dev, host64, sync_ok
from serving_refs import Paged, VALUES, attention_tolerance

pytestmark = pytest.mark.gpu

# heads, KV heads, head_dim, shards: own KV heads a shard, replicated ones, odd groups, one head.
GEOMETRIES = [(8, 2, 128, 2), (16, 2, 64, 8), (6, 2, 128, 1), (4, 4, 64, 4), (5, 1, 64, 1), (32, 8, 128, 8)]
LENS = {
    "single": [(1, 1)],
    "decode": [(1, 1), (1, 15), (1, 16), (1, 17), (1, 64), (1, 129), (1, 300)],
    "drafted": [(3, 3), (5, 70), (2, 131), (4, 64)],
    "chunks": [(40, 40), (33, 200), (1, 77)],
    "odd": [(0, 9), (1, 0), (4, 2), (0, 0), (2, 33)],  # nothing new, nothing kept, more new than kept
}


def stored(cache):
    x = cache.tensors
    return [t.view(torch.int16).cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()
            for t in x[:4 if cache.kv_dtype == tp.TP_KV_E4M3 else 2]]


def same(got, want):
    return all(np.array_equal(g, w, equal_nan=g.dtype == np.float32) for g, w in zip(got, want))


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("geo,page", [(GEOMETRIES[0], 16), (GEOMETRIES[1], 64), (GEOMETRIES[2], 32), (GEOMETRIES[3], 128)])
def test_write_is_bit_exact(geo, page, kv, lens):
    x = Paged(*geo, page, LENS[lens], kv, seed=3, pad=2, first=1)
    plan, cache = x.upload()
    tp.tp_kv_cache_write(plan, cache, dev(x.QKV))
    sync_ok(plan)
    K, V, ks, vs = x.written()
    assert same(stored(cache), [K, V] if kv == "bf16" else [K, V, ks, vs])


def test_write_quantises_edge_values():
    x = Paged(4, 4, 64, 1, 16, [(9, 9)], "e4m3", seed=4)
    v = x.QKV
    v[0] = 0
    v[1] *= 2.0 ** -130                 # below the least amax
    v[2, 260] = float("inf")
    v[3, 261] = float("nan")
    v[4] = 3.3895313892515355e38
    v[5, 256:320] = 0
    v[5, 300] = -1e-40                  # a subnormal alone
    v[6] = float("-inf")
    v[7] = float("nan")
    plan, cache = x.upload()
    tp.tp_kv_cache_write(plan, cache, dev(v))
    sync_ok(plan)
    assert same(stored(cache), [y for y in (x.written()[i] for i in (0, 1, 2, 3))])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("geo,page", [(GEOMETRIES[0], 64), (GEOMETRIES[1], 16), (GEOMETRIES[3], 128)])
def test_read_back(geo, page, kv):
    x = Paged(*geo, page, [(1, 5), (1, 64), (0, 0), (1, 131), (1, 16)], kv, seed=5)
    plan, cache = x.upload()
    cache.q_start = None                # reading needs no rows
    for max_len in (131, 64, 1):
        K, V = (torch.full((x.n_seqs, max_len, x.k, x.d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        tp.tp_kv_cache_read(plan, cache, max_len, K, V)
        sync_ok(plan)
        for got, part in ((K, "K"), (V, "V")):
            for s in range(x.n_seqs):
                n = min(x.len[s], max_len)
                # code * scale in fp32, rounded once to bf16: both steps redone here.
                want = torch.from_numpy(x.cached(part, s)[:n]).float().to(torch.bfloat16)
                assert torch.equal(got[s, :n].cpu(), want)
                assert bool((got[s, n:] == 7).all())


def attend(x, max_new=None, plan_cache=None):
    plan, cache = plan_cache or x.upload(max_new)
    n = tp.tp_plan_workspace_bytes(plan, tp.TP_OP_ATTN_PAGED)
    ws = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda")  # NaN to whoever reads it unprepared
    O = torch.full((x.rows, x.a * x.d), 7.0, dtype=torch.bfloat16, device="cuda")
    tp.tp_attn_paged_forward(plan, cache, dev(x.QKV), O, ws, n)
    return plan, O


def check_attention(x, O):
    want, A, E = x.attention()
    got = host64(O).reshape(x.rows, x.a, x.d)
    own = x.owned()
    assert (got[~own] == 7).all()
    err = np.abs(got - want)[own]
    tol = attention_tolerance(want, A, E)[own]
    assert np.isfinite(got[own]).all()
    assert (err <= tol).all(), f"worst {np.max(err / np.maximum(tol, 1e-30)):.2f} of the tolerance"


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("geo,page", [(GEOMETRIES[0], 16), (GEOMETRIES[1], 64), (GEOMETRIES[2], 32), (GEOMETRIES[3], 128),
                                      (GEOMETRIES[4], 16), (GEOMETRIES[5], 64)])
def test_attention(geo, page, kv, lens):
    x = Paged(*geo, page, LENS[lens], kv, seed=6, pad=2, first=1)
    for max_new in (None, 0, 1):        # the hint chooses the kernel alone
        plan, O = attend(x, max_new)
        sync_ok(plan)
        check_attention(x, O)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens", [[(1, 5000)], [(1, 2500), (3, 1), (1, 900)], [(70, 1500)], [(130, 130), (140, 800)]])
def test_attention_split_over_long_sequences(kv, lens):
    x = Paged(8, 2, 128, 2, 64, lens, kv, seed=7)
    plan, O = attend(x)
    sync_ok(plan)
    check_attention(x, O)


# Long sequences' chunks between single tokens: from 8 bits a launch for each, the sequences told apart on the GPU.
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("geo,page", [((8, 2, 128, 2), 64), ((16, 1, 64, 1), 16), ((6, 2, 64, 2), 128), ((32, 2, 128, 2), 32)])
@pytest.mark.parametrize("lens", [[(1, 1200), (50, 300), (0, 40), (2, 700), (3, 2), (1, 1), (9, 9), (1, 64)],
                                  [(1, 1100)] * 5 + [(33, 40)], [(40, 1050), (0, 0), (0, 9), (0, 3)],
                                  [(0, 0)] + [(1, 30)] * 300 + [(17, 1030)]])
def test_attention_of_a_mixture(geo, page, kv, lens):
    x = Paged(*geo, page, lens, kv, seed=12, pad=3, first=2)
    plan, O = attend(x)
    sync_ok(plan)
    check_attention(x, O)


def test_attention_of_many_sequences():
    rng = np.random.default_rng(8)
    lens = [(int(n), int(n + c)) for n, c in zip(rng.integers(0, 3, 700), rng.integers(0, 40, 700))]
    x = Paged(4, 2, 64, 2, 16, lens, seed=9)
    plan, O = attend(x)
    sync_ok(plan)
    check_attention(x, O)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_attention_large_scores(kv):
    # Scores of hundreds: the running maximum moves late and far.
    x = Paged(8, 2, 64, 2, 16, [(1, 400), (20, 260)], kv, seed=10, scale=6.0)
    plan, O = attend(x)
    sync_ok(plan)
    want, A, E = x.attention()
    got = host64(O).reshape(x.rows, x.a, x.d)
    # sum |q k| / sqrt d is up to about 40 times that of standard normal values here, and with it the
    # scores' share of the tolerance: 2^-12 * 2^6.
    worst = (np.abs(got - want) / (attention_tolerance(want, A, E) + 2.0 ** -6 * A + 1e-300)).max()
    assert worst <= 1, worst


def test_attention_repeats_bit_for_bit():
    x = Paged(8, 2, 128, 2, 64, [(1, 3000), (3, 700), (60, 400)], seed=11)
    pc = x.upload()
    first = attend(x, plan_cache=pc)[1].clone()
    for _ in range(3):
        assert torch.equal(attend(x, plan_cache=pc)[1], first)


@pytest.mark.parametrize("geo,page,lens", [((24, 4, 128, 2), 32, [(3, 2000 + 7 * i) for i in range(48)]),
                                           ((16, 2, 64, 1), 16, [(1 + i % 6, 900 + 61 * i) for i in range(40)]),
                                           ((8, 4, 128, 1), 64, [(17, 1000 + 33 * i) for i in range(12)])])
def test_many_short_tiles_repeat_bit_for_bit(geo, page, lens):
    # Many tiles a CTA, each with a ragged last block, whose rows of V behind the last key are cleared while the
    # next blocks' loads are on their way: every run gives the same bits, and right ones.
    x = Paged(*geo, page, [(n, m) for n, m in lens[:6]], seed=26)
    for y in (x, None):
        if y is None:               # too many to check against float64: the runs against each other
            y = Paged(*geo, page, lens, seed=27)
        plan, cache = y.upload()
        QKV = dev(y.QKV)
        n = tp.tp_plan_workspace_bytes(plan, tp.TP_OP_ATTN_PAGED)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        O = [torch.full((y.rows, y.a * y.d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        tp.tp_attn_paged_forward(plan, cache, QKV, O[0], ws, n)
        wrong = torch.zeros((), dtype=torch.int64, device="cuda")
        for _ in range(300):
            tp.tp_attn_paged_forward(plan, cache, QKV, O[1], ws, n)
            wrong += (O[0].view(torch.int16) != O[1].view(torch.int16)).sum()
        sync_ok(plan)
        assert int(wrong) == 0
        if y is x:
            check_attention(x, O[0])


def test_pages_shared_by_sequences():
    x = Paged(8, 2, 64, 2, 16, [(1, 60), (1, 50)], seed=12)
    x.table[1, :2] = x.table[0, :2]     # a common beginning of 32 tokens
    plan, O = attend(x)
    sync_ok(plan)
    check_attention(x, O)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_pages_outside_the_cache(kv):
    x = Paged(8, 2, 64, 2, 16, [(2, 60), (1, 50), (1, 70)], kv, seed=13)
    x.table[0, 1], x.table[1, 0], x.table[2, 2] = -5, x.n_pages, 2 ** 31 - 1
    x.table[2, 4] = -1                  # the new token's own page
    plan, cache = x.upload()
    tp.tp_kv_cache_write(plan, cache, dev(x.QKV))
    torch.cuda.synchronize()
    assert tp.tp_get_device_status(plan) == tp.TP_ERR_INVALID_ARG
    assert tp.tp_get_device_status(plan) == tp.TP_OK        # read and cleared
    K, V, ks, vs = x.written()
    assert same(stored(cache), [K, V] if kv == "bf16" else [K, V, ks, vs])
    _, cache = x.upload()
    plan, O = attend(x, plan_cache=(plan, cache))
    torch.cuda.synchronize()
    assert tp.tp_get_device_status(plan) == tp.TP_ERR_INVALID_ARG
    check_attention(x, O)               # keys without a page count as zeros
    out = [torch.full((3, 70, x.k, x.d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    tp.tp_kv_cache_read(plan, cache, 70, *out)
    torch.cuda.synchronize()
    assert tp.tp_get_device_status(plan) == tp.TP_ERR_INVALID_ARG
    for s in range(3):
        assert torch.equal(out[0][s, :x.len[s]].cpu(), torch.from_numpy(x.cached("K", s)).float().to(torch.bfloat16))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[(1, 300), (1, 80), (2, 40)], [(20, 300), (20, 80), (33, 200)]])
def test_scales_of_zero(d, lens):
    # A row of an 8-bit cache may hold a scale of zero (its values are zeros, whatever the codes), and all the rows of a
    # sequence may, or have no page.
    x = Paged(8, 2, d, 2, 16, lens, "e4m3", seed=22)
    g = torch.Generator().manual_seed(23)
    for sc in (x.ks, x.vs):
        sc[torch.rand(sc.shape, generator=g) < 0.3] = 0
    x.vs[x.table[1, :5]] = 0
    x.table[2] = -1
    plan, O = attend(x)
    torch.cuda.synchronize()
    assert tp.tp_get_device_status(plan) == tp.TP_ERR_INVALID_ARG
    check_attention(x, O)


def test_positions_past_the_page_table():
    x = Paged(8, 2, 64, 2, 16, [(1, 30), (1, 20)], seed=14)
    plan, cache = x.upload()
    cache.tensors[-1].copy_(torch.tensor([45, 20], dtype=torch.int32))   # kv_len: the table has 32 positions
    x.len[0] = 45
    tp.tp_kv_cache_write(plan, cache, dev(x.QKV))
    torch.cuda.synchronize()
    assert tp.tp_get_device_status(plan) == tp.TP_ERR_INVALID_ARG
    assert same(stored(cache), x.written()[:2])


def test_captured_call_follows_the_lengths():
    x = Paged(8, 2, 128, 2, 16, [(1, 40), (1, 90)], seed=15)
    y = Paged(8, 2, 128, 2, 16, [(1, 40), (1, 90)], seed=15)
    plan, cache = x.upload()
    QKV = dev(x.QKV)
    n = tp.tp_plan_workspace_bytes(plan, tp.TP_OP_ATTN_PAGED)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    O = torch.zeros(x.rows, x.a * x.d, dtype=torch.bfloat16, device="cuda")

    def step():
        tp.tp_kv_cache_write(plan, cache, QKV)
        tp.tp_attn_paged_forward(plan, cache, QKV, O, ws, n)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([40, 90], [33, 81], [12, 90]):     # shorter: rows already there are rewritten
        cache.tensors[-1].copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        sync_ok(plan)
        y.len = lens
        K, V = (torch.from_numpy(t).view(torch.bfloat16) for t in y.written()[:2])
        y.K, y.V = K, V
        check_attention(y, O)


def test_two_graphs_at_once():
    # Each with a workspace of its own, replayed on two streams: a mixture (two pairs of launches) and single tokens.
    calls = []
    for lens, seed in (([(1, 1100), (30, 400), (1, 900), (0, 0), (1, 30)], 24), ([(1, 700), (1, 1300), (1, 5)], 25)):
        x = Paged(8, 2, 128, 2, 64, lens, "e4m3", seed=seed)
        plan, cache = x.upload()
        n = tp.tp_plan_workspace_bytes(plan, tp.TP_OP_ATTN_PAGED)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        QKV, O = dev(x.QKV), torch.full((x.rows, x.a * x.d), 7.0, dtype=torch.bfloat16, device="cuda")
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        tp.tp_attn_paged_forward(plan, cache, QKV, O, ws, n)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            for _ in range(4):
                tp.tp_attn_paged_forward(plan, cache, QKV, O, ws, n)
        O.fill_(7.0)
        calls.append((x, plan, O, graph, side, cache, QKV, ws))
    torch.cuda.synchronize()
    for _ in range(5):
        for _, _, _, graph, side, *_ in calls:
            with torch.cuda.stream(side):
                graph.replay()
    torch.cuda.synchronize()
    for x, plan, O, *_ in calls:
        sync_ok(plan)
        check_attention(x, O)


def test_on_another_stream():
    x = Paged(8, 2, 64, 2, 16, [(1, 200), (4, 90)], seed=16)
    plan, cache = x.upload()
    QKV = dev(x.QKV)
    n = tp.tp_plan_workspace_bytes(plan, tp.TP_OP_ATTN_PAGED)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    O = torch.full((x.rows, x.a * x.d), 7.0, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    tp.tp_attn_paged_forward(plan, cache, QKV, O, ws, n, stream=side)
    side.synchronize()
    assert tp.tp_get_device_status(plan, side) == tp.TP_OK
    check_attention(x, O)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_offsets_past_32_bits(kv):
    # Pages whose elements lie past 2^31 (and whose bytes lie past 2^32 in bf16).
    x = Paged(8, 8, 128, 1, 128, [(2, 300)], kv, seed=17)
    plan, cache = x.upload()
    pages, shift = 17000, 16500
    big = [torch.zeros((pages,) + t.shape[1:], dtype=t.dtype, device="cuda") for t in cache.tensors[:-3]]
    for b, t in zip(big, cache.tensors):
        b[shift:shift + x.n_pages] = t
    table = cache.tensors[-3] + shift
    scales = dict(k_scale=big[2], v_scale=big[3]) if kv == "e4m3" else {}
    far = tp.make_kv_cache(big[0], big[1], table, cache.tensors[-2], cache.tensors[-1], max_new=2, **scales)
    plan, O = attend(x, plan_cache=(plan, far))
    sync_ok(plan)
    check_attention(x, O)
    tp.tp_kv_cache_write(plan, far, dev(x.QKV))
    sync_ok(plan)
    got = [b[shift:shift + x.n_pages] for b in big]
    got = [t.view(torch.int16).cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy() for t in got]
    K, V, ks, vs = x.written()
    assert same(got, [K, V] if kv == "bf16" else [K, V, ks, vs])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_batch_of_no_sequences(kv):
    # Nothing is written or read; the block still computes the rows that no sequence owns.
    x = Paged(8, 2, 64, 2, 16, [(2, 20)], kv, seed=28)
    plan, full = x.upload()
    scales = dict(zip(("k_scale", "v_scale"), full.tensors[2:4])) if kv == "e4m3" else {}
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    cache = tp.make_kv_cache(full.tensors[0], full.tensors[1], i32(0, 4), i32(1), i32(0), **scales)
    before = stored(full)
    tp.tp_kv_cache_write(plan, cache, dev(x.QKV))
    out = torch.zeros(0, 5, x.k, x.d, dtype=torch.bfloat16, device="cuda")
    tp.tp_kv_cache_read(plan, cache, 5, out, out)
    tp.tp_kv_cache_read(plan, full, 0, out, out)
    plan, O = attend(x, plan_cache=(plan, cache))
    assert (O == 7).all() and same(stored(full), before)
    h = 64
    W = [dev(synth.normal_bf16(s, 0.1, 80 + i)) for i, s in enumerate([(x.a * x.d, h), (x.k * x.d, h), (x.k * x.d, h), (h, x.a * x.d)])]
    n = tp.tp_plan_workspace_bytes(plan, tp.TP_OP_ATTN_CACHED)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    X, y = dev(synth.normal_bf16((x.rows, h), 1.0, 90)), torch.empty(x.rows, h, dtype=torch.bfloat16, device="cuda")
    tp.tp_attn_cached_forward(plan, cache, X, *W, X, None, y, ws, n)
    sync_ok(plan)
    assert torch.equal(y, X)            # the residual, and o_proj of zeros
    assert same(stored(full), before)


def test_refusals():
    x = Paged(8, 2, 64, 2, 16, [(1, 20)], seed=18)
    plan, cache = x.upload()
    n = tp.tp_plan_workspace_bytes(plan, tp.TP_OP_ATTN_PAGED)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    QKV, O = dev(x.QKV), torch.zeros(x.rows, x.a * x.d, dtype=torch.bfloat16, device="cuda")

    def code(fn, *args):
        with pytest.raises(tp.TPError) as e:
            fn(*args)
        return e.value.code

    assert code(tp.tp_attn_paged_forward, plan, cache, None, O, ws, n) == tp.TP_ERR_INVALID_ARG
    assert code(tp.tp_attn_paged_forward, plan, cache, QKV, None, ws, n) == tp.TP_ERR_INVALID_ARG
    if n:
        assert code(tp.tp_attn_paged_forward, plan, cache, QKV, O, ws, n - 1) == tp.TP_ERR_WORKSPACE
        assert code(tp.tp_attn_paged_forward, plan, cache, QKV, O, None, n) == tp.TP_ERR_WORKSPACE
    assert code(tp.tp_kv_cache_write, plan, cache, None) == tp.TP_ERR_INVALID_ARG
    assert code(tp.tp_kv_cache_read, plan, cache, -1, O, O) == tp.TP_ERR_INVALID_ARG
    cache.page_size = 8
    assert code(tp.tp_kv_cache_write, plan, cache, QKV) == tp.TP_ERR_UNSUPPORTED
    cache.page_size = 16
    cache.kv_heads = 1
    assert code(tp.tp_attn_paged_forward, plan, cache, QKV, O, ws, n) == tp.TP_ERR_INVALID_ARG
    mlp = tp.Plan(tp.make_config(tokens=4, hidden=64, ffn=64))
    assert code(tp.tp_kv_cache_write, mlp, cache, QKV) == tp.TP_ERR_INVALID_ARG
    wide = Paged(129, 1, 64, 1, 16, [(1, 3)])
    p2, c2 = wide.upload()
    assert code(tp.tp_attn_paged_forward, p2, c2, dev(wide.QKV), O, ws, n) == tp.TP_ERR_UNSUPPORTED
    assert tp.tp_get_device_status(plan) == tp.TP_OK


@pytest.mark.parametrize("mode", [tp.TP_REDUCE_FUSED, tp.TP_REDUCE_PARTIALS])
@pytest.mark.parametrize("a,k,d,t,kv", [(8, 2, 64, 4, "bf16"), (8, 4, 128, 2, "bf16"), (8, 4, 128, 2, "e4m3")])
def test_block_in_pieces_is_the_block_at_once(a, k, d, t, kv, mode):
    """Two prompts through tp_attn_cached_forward in pieces (a chunk, single tokens, drafts of which
    some are dropped again), against the 64-bit attention block of the whole prompts."""
    h, total, page = 128, [37, 50], 16
    X = [synth.normal_bf16((n, h), 1.0, 40 + n) for n in total]
    W = {n: synth.normal_bf16(s, 0.08, 50 + i) for i, (n, s) in enumerate(
        {"Wq": (a * d, h), "Wk": (k * d, h), "Wv": (k * d, h), "Wo": (h, a * d)}.items())}
    want = [oracle.attention(1, n, a, k, d, *(host64(v) for v in (X[s], W["Wq"], W["Wk"], W["Wv"], W["Wo"])))
            for s, n in enumerate(total)]
    # (rows of each sequence in a call, rows kept); the plan has room for 24 rows.
    calls = [((17, 0), (17, 0)), ((1, 20), (1, 20)), ((4, 1), (2, 1)), ((0, 5), (0, 3)), ((17, 6), (17, 6)),
             ((0, 20), (0, 20))]
    M = 24
    plan = tp.Plan(tp.make_config(tokens=M, hidden=h, n_heads=a, n_kv_heads=k, head_dim=d, tp_degree=t, reduce_mode=mode))
    dt = torch.bfloat16 if kv == "bf16" else torch.uint8
    K, V = (torch.zeros(8, k, page, d, dtype=dt, device="cuda") for _ in range(2))
    scales = {} if kv == "bf16" else {n: torch.zeros(8, k, page, device="cuda") for n in ("k_scale", "v_scale")}
    table = torch.tensor([[5, 0, 7, -1], [2, 6, 1, 3]], dtype=torch.int32, device="cuda")
    q_start, kv_len = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    cache = tp.make_kv_cache(K, V, table, q_start, kv_len, **scales)
    n = tp.tp_plan_workspace_bytes(plan, tp.TP_OP_ATTN_CACHED)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    wd = {n_: dev(v) for n_, v in W.items()}
    partials = torch.empty(t, M, h, device="cuda")
    done = [0, 0]
    for rows, kept in calls:
        x = torch.full((M, h), float("nan"), dtype=torch.bfloat16)   # rows of nobody
        x[:rows[0]] = X[0][done[0]:done[0] + rows[0]]
        x[rows[0]:sum(rows)] = X[1][done[1]:done[1] + rows[1]]
        q_start.copy_(torch.tensor([0, rows[0], sum(rows)], dtype=torch.int32))
        kv_len.copy_(torch.tensor([done[0] + rows[0], done[1] + rows[1]], dtype=torch.int32))
        cache.max_new = max(rows)
        res = torch.zeros(M, h, dtype=torch.bfloat16)
        res[sum(rows):] = 3
        out = torch.empty(M, h, dtype=torch.bfloat16, device="cuda")
        tp.tp_attn_cached_forward(plan, cache, dev(x), wd["Wq"], wd["Wk"], wd["Wv"], wd["Wo"], dev(res),
                                  partials if mode == tp.TP_REDUCE_PARTIALS else None, out, ws, n)
        sync_ok(plan)
        got = host64(out)
        assert (got[sum(rows):] == 3).all()
        at = 0
        for s in (0, 1):
            ref = want[s][done[s]:done[s] + rows[s]]
            # The framework's parity bar for bf16; 8-bit keys and values are off by half a step, 2^-4 of
            # each value, at random: over d = 128 terms and the block's averaging that is a few per cent
            # of the largest output, held to four times the bar.
            tol = 2e-2 if kv == "bf16" else 8e-2
            assert np.abs(got[at:at + rows[s]] - ref).max(initial=0) <= tol * np.abs(want[s]).max()
            at += rows[s]
            done[s] += kept[s]
    assert done == total
