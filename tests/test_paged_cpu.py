"""CPU checks of the paged cache: refusals of its host-only validation, and the index arithmetic that
the kernels run (csrc/tp_paged_index.h), compiled for the host and compared with plain loops, bad
pages and bad row numbers among the inputs."""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest
import torch

import megatron_tensor_transformer_colwise_gb300 as tp
from serving_refs import Paged, quantise, VALUES

CSRC = os.path.join(os.path.dirname(os.path.abspath(tp.__file__)), "csrc")


def config(**kw):
    base = dict(tokens=8, hidden=64, n_heads=8, n_kv_heads=2, head_dim=64, tp_degree=4)
    base.update(kw)
    return tp.make_config(**base)


def cache(kv_dtype=tp.TP_KV_BF16, **kw):
    # Addresses are only looked at for alignment here.
    scaled = kv_dtype == tp.TP_KV_E4M3
    f = dict(K=1 << 20, V=2 << 20, k_scale=3 << 20 if scaled else None, v_scale=4 << 20 if scaled else None,
             page_table=5 << 20, q_start=6 << 20, kv_len=7 << 20, n_pages=10, n_seqs=3, max_pages=4, page_size=16,
             kv_dtype=kv_dtype, kv_heads=2, head_dim=64, max_new=1)
    f.update(kw)
    return tp.TPKVCache(**f)


@pytest.mark.parametrize("cfg,kw,want", [
    ({}, {}, tp.TP_OK),
    ({}, dict(kv_dtype=tp.TP_KV_E4M3), tp.TP_OK),
    ({}, dict(n_seqs=0), tp.TP_OK),
    ({}, dict(max_new=0), tp.TP_OK),
    ({}, dict(n_pages=0x7fffffff), tp.TP_OK),
    (dict(n_heads=0, n_kv_heads=0, head_dim=0, ffn=64), {}, tp.TP_ERR_INVALID_ARG),
    (dict(n_heads=6), {}, tp.TP_ERR_NOT_DIVISIBLE),
    ({}, dict(K=None), tp.TP_ERR_INVALID_ARG),
    ({}, dict(V=(2 << 20) + 8), tp.TP_ERR_INVALID_ARG),
    ({}, dict(page_table=None), tp.TP_ERR_INVALID_ARG),
    ({}, dict(kv_len=None), tp.TP_ERR_INVALID_ARG),
    ({}, dict(q_start=None), tp.TP_ERR_INVALID_ARG),
    ({}, dict(kv_heads=4), tp.TP_ERR_INVALID_ARG),
    ({}, dict(head_dim=128), tp.TP_ERR_INVALID_ARG),
    ({}, dict(kv_dtype=2), tp.TP_ERR_INVALID_ARG),
    ({}, dict(k_scale=3 << 20), tp.TP_ERR_INVALID_ARG),
    ({}, dict(kv_dtype=tp.TP_KV_E4M3, v_scale=None), tp.TP_ERR_INVALID_ARG),
    ({}, dict(n_seqs=-1), tp.TP_ERR_INVALID_ARG),
    ({}, dict(page_size=8), tp.TP_ERR_UNSUPPORTED),
    ({}, dict(page_size=48), tp.TP_ERR_UNSUPPORTED),
    ({}, dict(page_size=256), tp.TP_ERR_UNSUPPORTED),
    ({}, dict(n_pages=0), tp.TP_ERR_INVALID_ARG),
    ({}, dict(n_pages=1 << 31), tp.TP_ERR_INVALID_ARG),
    ({}, dict(max_pages=0), tp.TP_ERR_INVALID_ARG),
    ({}, dict(max_pages=1 << 27), tp.TP_ERR_INVALID_ARG),
    ({}, dict(max_new=-1), tp.TP_ERR_INVALID_ARG),
])
def test_cache_check(cfg, kw, want):
    assert tp.tp_kv_cache_check(config(**cfg), cache(**kw)) == want, tp.tp_last_error()


def test_a_batch_of_no_sequences_is_a_batch():
    # Tensors without elements have no address.
    K, i = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16), lambda *s: torch.zeros(*s, dtype=torch.int32)
    c = tp.make_kv_cache(K, K.clone(), i(0, 4), i(1), i(0))
    assert c.page_table is None and c.kv_len is None
    c.q_start = 1 << 20                 # (alignment of host tensors aside)
    c.K, c.V = 1 << 21, 1 << 22
    for rows in (True, False):
        assert tp.tp_kv_cache_check(config(), c, rows) == tp.TP_OK, tp.tp_last_error()
    c.n_seqs = 1
    assert tp.tp_kv_cache_check(config(), c) == tp.TP_ERR_INVALID_ARG
    assert tp.tp_kv_cache_check(config(), cache(n_seqs=0, kv_len=4)) == tp.TP_ERR_INVALID_ARG  # misaligned


def test_cache_check_without_rows():
    assert tp.tp_kv_cache_check(config(), cache(q_start=None), needs_rows=False) == tp.TP_OK


def test_entry_points_refuse_null_plans_and_bad_vocabularies():
    L, c = tp.lib(), cache()
    assert L.tp_kv_cache_write(None, C.byref(c), None, None) == tp.TP_ERR_INVALID_ARG
    assert L.tp_kv_cache_read(None, C.byref(c), 4, None, None, None) == tp.TP_ERR_INVALID_ARG
    assert L.tp_attn_paged_forward(None, C.byref(c), None, None, None, 0, None) == tp.TP_ERR_INVALID_ARG
    assert L.tp_attn_cached_forward(None, C.byref(c), *([None] * 9), 0, None) == tp.TP_ERR_INVALID_ARG
    p = 1 << 20

    def verify(v=64, t=4, n=2, M=5, u=p, logits=p, tokens=p):
        return L.tp_vocab_verify_drafts(logits, None, M, v, t, p, p, n, None, u, None, p, tokens, None)

    assert verify(v=66) == tp.TP_ERR_NOT_DIVISIBLE
    assert verify(v=48) == tp.TP_ERR_INVALID_ARG       # 12 columns a shard
    assert verify(t=0) == tp.TP_ERR_INVALID_ARG
    assert verify(n=-1) == tp.TP_ERR_INVALID_ARG
    assert verify(M=-1) == tp.TP_ERR_INVALID_ARG
    assert verify(u=None) == tp.TP_ERR_INVALID_ARG
    assert verify(logits=p + 2) == tp.TP_ERR_INVALID_ARG
    assert verify(tokens=p + 4) == tp.TP_ERR_INVALID_ARG


def test_make_kv_cache_refuses_what_the_struct_cannot_say():
    K = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    args = dict(K=K, V=K.clone(), page_table=i(2, 4), q_start=i(3), kv_len=i(2))
    tp.make_kv_cache(**args)
    for bad in (dict(V=K[:2]), dict(V=K.float()), dict(K=K.float(), V=K.float()), dict(q_start=i(2)),
                dict(page_table=i(3, 4)), dict(kv_len=torch.zeros(2)), dict(k_scale=torch.zeros(3, 2, 16)),
                dict(page_table=i(4, 2).T), dict(K=K.to(torch.float8_e4m3fn), V=K.to(torch.float8_e4m3fn)),
                dict(K=K.byte(), V=K.byte(), k_scale=torch.zeros(3, 2, 8), v_scale=torch.zeros(3, 2, 16))):
        with pytest.raises(ValueError):
            tp.make_kv_cache(**{**args, **bad})


def test_quantise_reference_against_torch():
    x = torch.randn(200, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    x[3] = 0
    x[4, 5] = float("inf")
    x[5, 6] = float("nan")
    x[6] *= 2.0 ** -120
    code, scale = quantise(x.double().numpy())
    amax = x.float().abs().nan_to_num(0, float("inf")).amax(1).clamp(2.0 ** -100, 3.3895313892515355e38)
    back = torch.full_like(amax, 448) / amax
    y = (x.float() * back[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert np.array_equal(scale, (amax / 448).numpy())
    assert np.array_equal(code, y.view(torch.uint8).numpy())
    assert np.array_equal(VALUES, torch.arange(256).byte().view(torch.float8_e4m3fn).double().numpy(), equal_nan=True)


HOST = r"""
#include "tp_paged_index.h"
using namespace tpk;
static PagedView view(const int* table, const int* q, const int* len, long long pages, long long rows, int n,
                      int maxp, int log2, int k) {
    PagedView v{};
    v.table = table; v.q_start = q; v.kv_len = len; v.n_pages = pages; v.rows = rows;
    v.n_seqs = n; v.max_pages = maxp; v.page_log2 = log2; v.kv_heads = k; v.d = 64;
    return v;
}
extern "C" {
int owner(const int* q, int n, long long row) { return paged_owner(q, n, (int)row); }
void seq(const int* q, const int* len, long long rows, int n, int s, long long* out) {
    PagedSeq x = paged_seq(view(0, q, len, 0, rows, n, 0, 0, 1), s);
    out[0] = x.row0; out[1] = x.n; out[2] = x.len;
}
long long page(const int* table, long long pages, int maxp, int log2, int s, int pos) {
    return paged_page(view(table, 0, 0, pages, 0, 0, maxp, log2, 1), s, pos);
}
int least = 1, most = 0x7fffffff;
void take(int a, int b) { least = a; most = b; }
// The shares of a grid: for each block of work, in order, (sequence, g, tile, kb) into out, with the CTA
// and the slot its segment would be written to; desc as the kernel writes it.  Returns the total.
long long walk(const int* q, const int* len, long long rows, int n, int maxp, int log2, int k, int tok, int log2_keys,
               int G, int grid, int* out, long long cap, int* desc) {
    PagedView v = view(0, q, len, 1, rows, n, maxp, log2, k);
    Tiling t = {tok, G, log2_keys, exact_log2(tok), least, most};
    long long total = 0, done = 0;
    for (int s = 0; s < n; ++s) total += seq_blocks(v, paged_seq(v, s), t);
    const long long per = (total + grid - 1) / grid;
    for (int c = 0; c < grid; ++c) {
        desc[4 * c + 3] = 0;
        const long long begin = pmin(c * per, total), count = pmin(per, total - begin);
        int s = 0;
        long long at = 0;
        if (count > 0)
            for (;; ++s) {
                const long long m = seq_blocks(v, paged_seq(v, s), t);
                if (begin < at + m) break;
                at += m;
            }
        TileWalk w;
        w.left = 0;
        if (count > 0) {
            // As the kernels find the tile, one at a time instead of 32.
            const PagedSeq x = paged_seq(v, s);
            const int keys = paged_keys(v, x), tiles = seq_tiles(x, t);
            const long long per_head = tiles_blocks(x, keys, t, tiles);
            long long off = begin - at;
            int g = 0, tile = 0;
            for (; off >= per_head; ++g) off -= per_head;
            while (tile + 1 < tiles && tiles_blocks(x, keys, t, tile + 1) <= off) ++tile;
            w.q = x; w.left = count; w.s = s; w.g = g; w.tile = tile; w.tiles = tiles; w.keys = keys;
            w.kb = (int)(off - tiles_blocks(x, keys, t, tile)); w.nkb = tile_blocks(x, keys, t, tile);
        }
        for (; w.left > 0; w.next(v, t)) {
            const int seg = w.segment();
            const bool b = w.kb == 0, e = w.kb + seg == w.nkb;
            for (int i = 0; i < seg; ++i, ++done) {
                if (done >= cap) return -1;
                int* o = out + 6 * done;
                o[0] = w.s; o[1] = w.g; o[2] = w.tile; o[3] = w.kb + i; o[4] = c; o[5] = b && e ? -1 : b ? 1 : 0;
            }
            if (b && !e) {
                const long long first = begin + count - seg;
                desc[4 * c] = w.s; desc[4 * c + 1] = w.g; desc[4 * c + 2] = w.tile;
                desc[4 * c + 3] = (int)((first + w.nkb - 1) / per) - c + 1;
            }
        }
    }
    return done == total ? total : -2;
}
long long blocks(int n, int len, int maxp, int tok, int log2_keys) {
    const int q[2] = {0, n};
    PagedView v = view(0, q, &len, 1, n, 1, maxp, 4, 1);
    return seq_blocks(v, paged_seq(v, 0), Tiling{tok, 1, log2_keys, exact_log2(tok)});
}
long long row(int k, int log2, long long page, int g, int pos) {
    return paged_row(view(0, 0, 0, 0, 0, 0, 0, log2, k), page, g, pos);
}
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    d = tmp_path_factory.mktemp("paged_index")
    (d / "host.cpp").write_text(HOST)
    so = str(d / "host.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(d / "host.cpp"), "-o", so], check=True)
    L = C.CDLL(so)
    L.page.restype = L.row.restype = C.c_longlong
    L.page.argtypes = [C.c_void_p, C.c_longlong, C.c_int, C.c_int, C.c_int, C.c_int]
    L.row.argtypes = [C.c_int, C.c_int, C.c_longlong, C.c_int, C.c_int]
    L.owner.argtypes = [C.c_void_p, C.c_int, C.c_longlong]
    L.walk.restype = L.blocks.restype = C.c_longlong
    L.walk.argtypes = [C.c_void_p, C.c_void_p, C.c_longlong] + [C.c_int] * 8 + [C.c_void_p, C.c_longlong, C.c_void_p]
    L.seq.argtypes = [C.c_void_p, C.c_void_p, C.c_longlong, C.c_int, C.c_int, C.c_void_p]
    return L


def i32(x):
    return np.ascontiguousarray(x, dtype=np.int32)


def test_owner_of_a_row(host):
    q = i32([2, 2, 5, 5, 5, 9, 9])
    for row in range(-1, 12):
        want = [s for s in range(6) if q[s] <= row < q[s + 1]]
        assert host.owner(q.ctypes.data, 6, row) == (want[0] if want else -1)
    assert host.owner(i32([0]).ctypes.data, 0, 0) == -1


def test_bad_row_numbers_are_clamped(host):
    rng = np.random.default_rng(0)
    out = np.zeros(3, dtype=np.int64)
    for _ in range(300):
        q, length = i32(rng.integers(-5, 30, 5)), i32(rng.integers(-2 ** 31, 2 ** 31, 4))
        for s in range(4):
            host.seq(q.ctypes.data, length.ctypes.data, 20, 4, s, out.ctypes.data)
            assert 0 <= out[0] and out[1] >= 0 and out[0] + out[1] <= 20 and 0 <= out[2] <= 1 << 30
        assert -1 <= host.owner(q.ctypes.data, 4, int(rng.integers(-2, 25))) < 4


def test_bad_pages_are_never_an_address(host):
    rng = np.random.default_rng(1)
    for log2 in (4, 5, 6, 7):
        table = i32(rng.choice([-2 ** 31, -1, 0, 1, 6, 7, 8, 2 ** 31 - 1], (3, 4)))
        for s in range(3):
            for pos in [-2 ** 31, -1, 0, 1, *rng.integers(0, 5 << log2, 40).tolist(), (4 << log2) - 1, 4 << log2, 2 ** 31 - 1]:
                i = pos >> log2
                want = int(table[s, i]) if 0 <= i < 4 and 0 <= table[s, i] < 7 else -1
                assert host.page(table.ctypes.data, 7, 4, log2, s, pos) == want


def test_cache_rows_pass_32_bits(host):
    assert host.row(8, 7, 2 ** 31 - 1, 7, 131) == ((2 ** 31 - 1) * 8 + 7) * 128 + 3
    assert host.row(2, 4, 5, 1, 35) == (5 * 2 + 1) * 16 + 3


@pytest.mark.parametrize("rows,log2_keys", [(16, 6), (16, 7), (128, 7)])
def test_shares_cover_all_work_once(host, rows, log2_keys):
    rng, KB = np.random.default_rng(rows + log2_keys), 1 << log2_keys
    for trial in range(100):
        n, k, G = int(rng.integers(1, 9)), int(rng.choice([1, 2, 3])), int(rng.choice([1, 3, 4, 5, 7, 8, 16]))
        tok = rows // G
        new, keep = rng.integers(0, 90, n), rng.integers(0, 900, n)
        if trial % 3 == 0:
            new = rng.integers(0, 3, n)
        length = i32(np.maximum(new + keep - (trial % 4 == 0) * 300, 0))   # some with more new than kept
        q, maxp = i32(np.cumsum([0, *new])), int(rng.integers(1, 80))
        grid = int(rng.choice([1, 2, 7, 152]))
        want = []
        for s in range(n):
            keys = min(int(length[s]), maxp * 16)
            for g in range(k):
                for tile in range(-(-int(new[s]) // tok)):
                    last = min((tile + 1) * tok, int(new[s])) - 1
                    seen = min(int(length[s]) - int(new[s]) + last + 1, keys)
                    want += [(s, g, tile, b) for b in range(max(1, -(-seen // KB)))]
        out, desc = np.zeros((len(want) + 1, 6), dtype=np.int32), np.zeros((grid, 4), dtype=np.int32)
        got = host.walk(q.ctypes.data, length.ctypes.data, int(q[-1]), n, maxp, 4, k, tok, log2_keys, G, grid, out.ctypes.data,
                        len(want), desc.ctypes.data)
        assert got == len(want)
        out = out[:got]
        assert [tuple(x) for x in out[:, :4].tolist()] == want
        # Parts: a tile cut by a share's border is in slot 1 of one CTA and slot 0 of the next ones.
        slots = {}
        for s, g, tile, b, cta, slot in out.tolist():
            slots.setdefault((s, g, tile), []).append((cta, slot))
        parts = 0
        for key, places in slots.items():
            places = sorted(set(places))
            if places[0][1] == -1:
                assert len(places) == 1
                continue
            c = places[0][0]
            assert places == [(c, 1)] + [(c + i, 0) for i in range(1, len(places))]
            assert desc[c].tolist() == [*key, len(places)]
            parts += 1
        assert (desc[:, 3] > 0).sum() == parts


def test_shares_of_some_sequences(host):
    # A launch that takes sequences of some numbers of new tokens alone: every block of those once, none of the others.
    rng = np.random.default_rng(77)
    try:
        for trial in range(60):
            n, k, bound = int(rng.integers(1, 12)), int(rng.choice([1, 3])), int(rng.choice([1, 2, 8]))
            new = np.where(rng.random(n) < 0.6, rng.integers(0, 4, n), rng.integers(0, 70, n))
            length = i32(new + rng.integers(0, 600, n))
            q, grid, both = i32(np.cumsum([0, *new])), int(rng.choice([1, 5, 152])), 0
            for least, most in ((1, bound), (bound + 1, 0x7fffffff)):
                tok = 4 if most == bound else 32
                want = [(s, g, tile, b) for s in range(n) if least <= new[s] <= most for g in range(k)
                        for tile in range(-(-int(new[s]) // tok))
                        for b in range(max(1, -(-(int(length[s]) - int(new[s]) + min((tile + 1) * tok, int(new[s]))) // 128)))]
                host.take(least, most)
                out, desc = np.zeros((len(want) + 1, 6), dtype=np.int32), np.zeros((grid, 4), dtype=np.int32)
                got = host.walk(q.ctypes.data, length.ctypes.data, int(q[-1]), n, 64, 4, k, tok, 7, 4, grid, out.ctypes.data,
                                len(want), desc.ctypes.data)
                assert got == len(want)
                assert [tuple(x) for x in out[:got, :4].tolist()] == want
                both += len({x[0] for x in want})
            assert both == (new > 0).sum()
    finally:
        host.take(1, 0x7fffffff)


def test_blocks_of_a_sequence_in_closed_form(host):
    """The sum over a sequence's tiles, against the loop: long sequences, ends of the page table inside."""
    rng = np.random.default_rng(5)
    out = np.zeros(1, dtype=np.int64)
    for _ in range(400):
        new, keep, tok = int(rng.integers(1, 5000)), int(rng.integers(-3000, 9000)), int(rng.choice([1, 2, 3, 5, 16, 18, 25, 32, 42, 64]))
        length, maxp, log2_keys = max(new + keep, 0), int(rng.integers(1, 900)), int(rng.choice([6, 7]))
        keys, want = min(length, 16 * maxp), 0
        for tile in range(-(-new // tok)):
            seen = min(length - new + min((tile + 1) * tok, new), keys)
            want += max(1, -(-seen >> log2_keys) if seen <= 0 else ((seen - 1) >> log2_keys) + 1)
        got = host.blocks(new, length, maxp, tok, log2_keys)
        assert got == want


def test_problems_own_their_rows():
    x = Paged(8, 2, 64, 4, 16, [(2, 20), (0, 5), (1, 1)], first=1, pad=2)
    assert x.rows == 6 and x.owned().tolist() == [False, True, True, True, False, False]
