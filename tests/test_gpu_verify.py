"""GPU tests of draft verification against its 64-bit definition."""
import numpy as np
import pytest
import torch

import megatron_tensor_transformer_colwise_gb300 as tp
from gpu_util import dev, sync_ok
from serving_refs import softmax64, verify

pytestmark = pytest.mark.gpu

# An fp32 probability is off by about 2^-24 (|x| / T log2 e + 8) of its value: below 1e-5 for the logits here
# (|x| / T up to 30).  A decision nearer to its border than that may go either way.
MARGIN = 2e-5


class Drafts:
    def __init__(self, rows, v, seed, T=(0.6, 1.3), greedy=0, near=0.5, pad=0, first=0):
        g = torch.Generator().manual_seed(seed)
        self.start = np.cumsum([first] + list(rows))
        M, n = int(self.start[-1]) + pad, len(rows)
        self.v = v
        self.logits = (torch.randn(M, v, generator=g) * 2.5).to(torch.bfloat16)
        self.draft = (self.logits.float() + torch.randn(M, v, generator=g) * near).to(torch.bfloat16)
        self.temperature = torch.rand(n, generator=g) * (T[1] - T[0]) + T[0]
        if greedy:
            self.temperature[::greedy] = 0
        self.ids = torch.randint(0, v, (M,), generator=g, dtype=torch.int32)
        for s in range(n):
            for r in range(self.start[s], self.start[s + 1] - 1):
                if self.temperature[s] > 0:
                    q = torch.from_numpy(softmax64(self.draft[r].double().numpy(), float(self.temperature[s])))
                    self.ids[r + 1] = int(torch.multinomial(q, 1, generator=g))
                else:
                    self.ids[r + 1] = int(self.draft[r].float().argmax())
        self.u = torch.rand(M, generator=g)
        self.noise = torch.empty(n, v).exponential_(generator=g)

    def run(self, t=1, draft=True, temperature=True, noise=True):
        M, n = self.logits.shape[0], len(self.start) - 1
        acc = torch.full((n,), -7, dtype=torch.int32, device="cuda")
        tok = torch.full((M,), -2, dtype=torch.int32, device="cuda")
        tp.tp_vocab_verify_drafts(dev(self.logits), dev(self.draft) if draft else None, M, self.v, t, dev(self.ids),
                                  dev(torch.as_tensor(self.start, dtype=torch.int32)), n,
                                  dev(self.temperature) if temperature else None, dev(self.u),
                                  dev(self.noise) if noise else None, acc, tok)
        sync_ok()
        return acc.cpu().numpy(), tok.cpu().numpy()

    def want(self, draft=True, temperature=True, noise=True):
        return verify(self.logits.double().numpy(), self.draft.double().numpy() if draft else None, self.ids.numpy(),
                      self.start, self.temperature.double().numpy() if temperature else None, self.u.double().numpy(),
                      self.noise.double().numpy() if noise else None)

    def check(self, least_clear=0.9, **kw):
        acc, tok = self.run(**kw)
        kw.pop("t", None)
        a, k, margin = self.want(**kw)
        clear = margin > MARGIN
        assert clear.mean() >= least_clear
        assert np.array_equal(acc[clear], a[clear])
        own = np.zeros(len(tok), dtype=bool)
        for s in range(len(a)):
            rows = slice(self.start[s], self.start[s + 1])
            own[rows] = True
            if clear[s]:
                assert np.array_equal(tok[rows], k[rows]), f"sequence {s}"
        assert (tok[~own] == -2).all()
        return a


@pytest.mark.parametrize("v,t", [(8, 1), (64, 2), (1000, 5), (4608, 8), (32768, 4)])
@pytest.mark.parametrize("rows", [[1], [4], [1, 5, 2, 0, 7, 3]])
def test_against_the_definition(v, t, rows):
    Drafts(rows, v, seed=v + len(rows), pad=2, first=1).check(t=t, least_clear=0.5)


@pytest.mark.parametrize("v", [8, 16, 56, 72])
def test_words_for_some_blocks_of_a_cluster_alone(v):
    # Blocks without words reach the exchange first, whatever the others do: every run gives the same, and right.
    d = Drafts([3, 1, 4] * 150, v, seed=v)
    d.check(least_clear=0.5)
    first = d.run()
    for _ in range(20):
        assert all(np.array_equal(a, b) for a, b in zip(d.run(), first))


def test_a_batch_takes_and_refuses():
    taken = Drafts([5] * 120, 1024, seed=5).check()
    assert 0 < taken.mean() < 4 and (taken == 4).any() and (taken == 0).any()


def test_long_drafts():
    taken = Drafts([70, 33, 9], 256, seed=6, near=0.02).check(least_clear=0.5)
    assert taken.max() > 16


@pytest.mark.parametrize("greedy", [1, 3])
def test_greedy(greedy):
    d = Drafts([4] * 40, 512, seed=7, greedy=greedy, near=0.3)
    taken = d.check()
    assert taken[::greedy].max() == 3
    # bf16 logits tie often: the first of the largest.
    d.logits[:, 100] = d.logits[:, 400] = 20.0
    d.check()
    assert (d.run()[1].reshape(40, 4)[::greedy][d.want()[0][::greedy] == 0][:, 0] == 100).all()


def test_without_draft_distribution_temperature_or_noise():
    d = Drafts([3, 1, 2], 128, seed=8)
    d.check(draft=False, least_clear=0.5)
    d.check(temperature=False, least_clear=0.5)
    d.check(noise=False, least_clear=0.5)
    d.temperature[:] = 0
    d.check(draft=False, noise=False)


def test_masked_and_hostile_logits():
    d = Drafts([2] * 12, 64, seed=9)
    lo = float("-inf")
    d.logits[0, 5:] = lo                       # a mask that leaves a few
    d.logits[2] = lo                           # nothing left at a draft
    d.logits[5] = lo                           # nothing left behind the draft
    d.draft[6] = lo                            # a draft distribution that is 0 everywhere
    d.logits[8] = torch.finfo(torch.bfloat16).min   # all equal, at the type's lowest value
    d.logits[10, 7] = 3e38                     # one huge
    d.ids[13], d.ids[15], d.ids[17] = -1, 64, 2 ** 31 - 1   # drafts outside the vocabulary
    d.temperature[9] = float("nan")            # greedy
    d.temperature[10] = -1.0                   # greedy
    d.u[4] = 0.0
    acc, tok = d.run()
    a, k, margin = d.want()
    clear = margin > MARGIN
    assert np.array_equal(acc[clear], a[clear])
    assert np.array_equal(tok.reshape(-1, 2)[clear], k.reshape(-1, 2)[clear])
    assert tok[2] == -1 and acc[1] == 0
    d.logits[0, 3] = float("nan")              # garbage in: an answer within range, no fault
    d.logits[2, 3] = float("inf")
    acc, tok = d.run()
    assert ((tok >= -1) & (tok < 64)).all() and ((acc >= 0) & (acc <= 1)).all()


def test_bad_row_numbers_are_clamped():
    d = Drafts([2, 2, 2], 64, seed=10)
    d.start = np.array([-4, 3, 2, 1 << 30])
    acc, tok = d.run()
    assert ((tok >= -2) & (tok < 64)).all() and ((acc >= 0) & (acc <= 6)).all()


def test_tokens_follow_the_target():
    """Speculation leaves the target's distribution as it is: the first settled token of 20,000
    sequences of one row pair, by a chi-square over the vocabulary."""
    v, n = 16, 20000
    d = Drafts([2], v, seed=11, T=(1, 1.0001), near=1.5)
    g = torch.Generator().manual_seed(12)
    q = torch.from_numpy(softmax64(d.draft[0].double().numpy(), 1.0))
    d.logits, d.draft = d.logits.repeat(n, 1), d.draft.repeat(n, 1)
    d.ids = torch.zeros(2 * n, dtype=torch.int32)
    d.ids[1::2] = torch.multinomial(q, n, replacement=True, generator=g).int()
    d.u, d.noise = torch.rand(2 * n, generator=g), torch.empty(n, v).exponential_(generator=g)
    d.start, d.temperature = np.arange(0, 2 * n + 1, 2), torch.ones(n)
    tok = d.run()[1][::2]
    p = softmax64(d.logits[0].double().numpy(), 1.0)
    big = p * n > 5
    count = np.bincount(tok, minlength=v)
    chi = ((count - n * p) ** 2 / (n * p))[big].sum()
    # Chi-square with at most 15 degrees of freedom: above 45 in fewer than one of 10,000 samples.
    assert chi < 45, chi


def test_infinite_temperature_is_uniform_over_what_is_left():
    # p and q are uniform over the words that are not masked; 1e300 says the same in 64 bits.
    d = Drafts([3, 1, 2, 4] * 20, 264, seed=32)
    lo = float("-inf")
    d.logits[::2, 40:] = lo
    d.logits[1::3, :30] = lo
    d.draft[::5, 100:200] = lo
    d.logits[3], d.logits[6, 7], d.logits[6, 8] = lo, 3e38, -3e38
    d.temperature[:] = float("inf")
    acc, tok = d.run()
    d.temperature = d.temperature.double()
    d.temperature[:] = 1e300
    a, k, margin = d.want()
    clear = margin > MARGIN
    assert clear.mean() > 0.5
    for s in np.flatnonzero(clear):
        assert acc[s] == a[s] and np.array_equal(tok[d.start[s]:d.start[s + 1]], k[d.start[s]:d.start[s + 1]]), s
    assert 0 < a.sum() and (k >= 0).mean() > 0.3


def test_infinite_temperature_counts_masks_of_the_lowest_value():
    # 0 times any finite logit is 0: words masked with bf16's lowest value are as likely as the others, so that p
    # and q are equal and every draft is taken.
    d = Drafts([3, 1, 2, 4] * 20, 264, seed=40)
    g = torch.Generator().manual_seed(41)
    for x in (d.logits, d.draft):
        x[torch.rand(x.shape, generator=g) < 0.4] = torch.finfo(torch.bfloat16).min
    d.logits[::4, 3], d.draft[::3, 9] = 3e38, 1e38
    d.u[::2] = 1 - 2.0 ** -22           # taken by a hair
    d.temperature[:] = float("inf")
    acc, tok = d.run()
    assert np.array_equal(acc, np.diff(d.start) - 1)
    want = torch.from_numpy(1 / d.noise.double().numpy()).argmax(1).numpy()
    assert np.array_equal(tok[d.start[1:] - 1], want)


@pytest.mark.parametrize("T", [1e-3, 1e-5, 1e-7, 1e-8, 3e-9, 1e-12, 1e-20, 1e-30, 1e-38])
def test_low_temperatures(T):
    # x / T goes up to 10^39: all but the largest logits vanish.  bf16 logits tie, so that drafts and draws among
    # equals are left to u and the noise.  A probability is off by 2^-22 (x_max - x) / T log2 e, which is below
    # 2 MARGIN where the probability itself is above 2^-80.
    d = Drafts([3, 1, 4, 2] * 30, 264, seed=33, near=0.1)
    g = torch.Generator().manual_seed(34)
    for x in (d.logits, d.draft):
        x += 20 * torch.randint(-1, 2, (x.shape[0], 1), generator=g)     # largest logits near 27, 7 and -13
        best = x.float().amax(1, keepdim=True).to(torch.bfloat16)
        x[:, 5:6] = x[:, 200:201] = best
    d.ids[:] = torch.where(torch.rand(len(d.ids), generator=g) < 0.5, 200, 5).int()
    d.temperature[:] = T
    taken = d.check(least_clear=0.9)
    assert taken.max() == 3 and taken.min() == 0


@pytest.mark.parametrize("where", [1, 2])
@pytest.mark.parametrize("v", [8, 1024, 128256])
def test_waits_that_give_up_leave_the_context_usable(v, where):
    # Waits that give up while copies are on their way: the kernel ends, and calls around it are right.
    d = Drafts([3, 1, 0, 5] * 10, v, seed=30)
    n, M = len(d.start) - 1, d.logits.shape[0]
    before = d.run(draft=False, temperature=False, noise=False)
    acc, tok = (torch.full((k,), -7, dtype=torch.int32, device="cuda") for k in (n, M))
    x = [dev(t) for t in (d.logits, d.ids, torch.as_tensor(d.start, dtype=torch.int32), d.u)]
    for _ in range(3):
        tp.tp_selftest_verify_timeout(x[0], M, v, x[1], x[2], n, x[3], acc, tok, where)
    sync_ok()
    after = d.run(draft=False, temperature=False, noise=False)
    assert all(np.array_equal(a, b) for a, b in zip(before, after))


@pytest.mark.parametrize("where", [1, 2])
@pytest.mark.parametrize("v", [8, 1024, 128256])
def test_a_wait_that_gives_up_settles_nothing(v, where):
    d = Drafts([3, 1, 0, 5, 40], v, seed=31, pad=2, first=1)
    n, M = len(d.start) - 1, d.logits.shape[0]
    acc, tok = (torch.full((k,), -7, dtype=torch.int32, device="cuda") for k in (n, M))
    tp.tp_selftest_verify_timeout(dev(d.logits), M, v, dev(d.ids), dev(torch.as_tensor(d.start, dtype=torch.int32)), n,
                                  dev(d.u), acc, tok, where)
    sync_ok()
    assert acc.tolist() == [-1, -1, 0, -1, -1]
    own = slice(int(d.start[0]), int(d.start[-1]))
    assert (tok[own] == -1).all()
    assert tok[0] == -7 and (tok[own.stop:] == -7).all()


def test_sequences_without_rows_alone():
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    acc, none = i32(3) - 7, i32(0)
    logits = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    tp.tp_vocab_verify_drafts(logits, logits, 0, 64, 2, none, i32(4), 3, None, none.float(),
                              torch.ones(3, 64, device="cuda"), acc, none)
    sync_ok()
    assert acc.tolist() == [0, 0, 0]
    tp.tp_vocab_verify_drafts(logits, None, 0, 64, 2, none, i32(1), 0, None, none.float(), None, none, none)
    d = Drafts([2, 1], 64, seed=35)     # rows of nobody
    tok = i32(3) - 2
    tp.tp_vocab_verify_drafts(dev(d.logits), dev(d.draft), 3, 64, 1, dev(d.ids), i32(1), 0, None, dev(d.u), None, none, tok)
    sync_ok()
    assert tok.tolist() == [-2, -2, -2]


def test_captured_and_replayed_with_new_numbers():
    d = Drafts([3, 2], 256, seed=13)
    n, M = 2, d.logits.shape[0]
    x = [dev(t) for t in (d.logits, d.draft, d.ids, torch.as_tensor(d.start, dtype=torch.int32), d.temperature, d.u, d.noise)]
    acc, tok = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(M, dtype=torch.int32, device="cuda")

    def step():
        tp.tp_vocab_verify_drafts(x[0], x[1], M, 256, 2, x[2], x[3], n, x[4], x[5], x[6], acc, tok)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (14, 15, 16):
        g = torch.Generator().manual_seed(seed)
        d.u, d.noise = torch.rand(M, generator=g), torch.empty(n, 256).exponential_(generator=g)
        x[5].copy_(d.u)
        x[6].copy_(d.noise)
        graph.replay()
        sync_ok()
        a, k, margin = d.want()
        if margin.min() > MARGIN:
            assert np.array_equal(acc.cpu().numpy(), a) and np.array_equal(tok.cpu().numpy(), k)


def test_decoding_with_drafts_is_decoding_without():
    """A toy language model (embedding, attention block over a cache, output layer) decodes greedily: with
    drafted tokens, right ones and wrong ones, it settles the tokens that single steps settle, up to the
    first place where two logits are so near that a bf16 rounding upstream may swap them."""
    import synth
    a, k, d, t, h, v, page = 4, 2, 64, 2, 128, 512, 16
    E = dev(synth.integer_bf16((v, h), -2, 2, 60))
    W = {n: dev(synth.normal_bf16(s, 0.1, 61 + i)) for i, (n, s) in enumerate(
        {"Wq": (a * d, h), "Wk": (k * d, h), "Wv": (k * d, h), "Wo": (h, a * d)}.items())}
    U = dev(synth.normal_bf16((v, h), 0.3, 70))
    table = torch.tensor([[3, 1, 4, 0]], dtype=torch.int32, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")

    class Model:
        def __init__(self):
            self.K, self.V = (torch.zeros(5, k, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            self.len = 0

        def step(self, ids):
            """Logits behind each of the new tokens (they enter the cache)."""
            M = len(ids)
            plan = tp.Plan(tp.make_config(tokens=M, hidden=h, n_heads=a, n_kv_heads=k, head_dim=d, tp_degree=t))
            n = tp.tp_plan_workspace_bytes(plan, tp.TP_OP_ATTN_CACHED)
            ws = torch.empty(n, dtype=torch.uint8, device="cuda")
            x, y = (torch.empty(M, h, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            logits = torch.empty(M, v, dtype=torch.bfloat16, device="cuda")
            cache = tp.make_kv_cache(self.K, self.V, table, i32(0, M), i32(self.len + M), max_new=M)
            tp.tp_vocab_embedding_forward(i32(*ids), M, E, v, h, t, x)
            tp.tp_attn_cached_forward(plan, cache, x, W["Wq"], W["Wk"], W["Wv"], W["Wo"], x, None, y, ws, n)
            tp.tp_vocab_logits_forward(y, M, h, U, v, t, logits)
            acc, tok = i32(0), torch.zeros(M, dtype=torch.int32, device="cuda")
            tp.tp_vocab_verify_drafts(logits, None, M, v, t, i32(*ids), i32(0, M), 1, torch.zeros(1, device="cuda"),
                                      torch.zeros(M, device="cuda"), None, acc, tok)
            sync_ok(plan)
            taken = int(acc)
            top = logits[taken].float().topk(2).values
            self.gap = float(top[0] - top[1])
            self.len += 1 + taken           # refused drafts leave the sequence again
            return tok.tolist()[:taken + 1]

    plain, text = Model(), [17]
    plain_text, sure = [17], 0
    while len(plain_text) < 50:
        plain_text += plain.step(plain_text[-1:])
        # One bf16 step of a logit near 16 is 2^-3, and the hidden state's own steps add about as much.
        if plain.gap > 0.5 and sure == len(plain_text) - 2:
            sure = len(plain_text) - 1
    fast, rng = Model(), np.random.default_rng(3)
    assert sure >= 6
    while len(text) + 6 < sure:
        right = int(rng.integers(0, 5))
        drafts = plain_text[len(text):len(text) + right]
        wrong = [(plain_text[min(len(text) + right, 49)] + 1) % v]
        got = fast.step(text[-1:] + drafts + wrong)
        assert len(got) == len(drafts) + 1
        text += got
    assert text == plain_text[:len(text)]


def test_every_replay_is_compared():
    d = Drafts([3, 1, 4, 2] * 10, 256, seed=36, greedy=5)
    n, M = len(d.start) - 1, d.logits.shape[0]
    x = [dev(t) for t in (d.logits, d.draft, d.ids, torch.as_tensor(d.start, dtype=torch.int32), d.temperature, d.u, d.noise)]
    acc, tok = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(M, dtype=torch.int32, device="cuda")

    def step():
        tp.tp_vocab_verify_drafts(x[0], x[1], M, 256, 2, x[2], x[3], n, x[4], x[5], x[6], acc, tok)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    seen = []
    for seed in (37, 38, 39):
        g = torch.Generator().manual_seed(seed)
        d.u, d.noise = torch.rand(M, generator=g), torch.empty(n, 256).exponential_(generator=g)
        x[5].copy_(d.u)
        x[6].copy_(d.noise)
        graph.replay()
        sync_ok()
        a, k, margin = d.want()
        clear = margin > MARGIN
        assert clear.mean() > 0.8
        assert np.array_equal(acc.cpu().numpy()[clear], a[clear])
        rows = np.repeat(clear, np.diff(d.start))
        assert np.array_equal(tok.cpu().numpy()[rows], k[rows])
        seen.append(tuple(k.tolist()))
    assert len(set(seen)) == 3              # each replay had answers of its own


def test_drafts_settle_what_single_steps_settle():
    """A toy language model (embedding, attention block over a cache, output layer) decodes 200 tokens greedily, one
    a step; then again with those as drafts and a wrong one behind them, refused drafts dropped from the
    cache.  Wherever the largest logit leads by more than roundings upstream move it, the drafted steps take the
    right drafts, refuse the wrong one and draw the same token."""
    import synth
    a, k, d, t, h, v, page, total = 4, 2, 64, 2, 128, 512, 16, 200
    E = dev(synth.integer_bf16((v, h), -2, 2, 60))
    W = [dev(synth.normal_bf16(s, 0.1, 61 + i)) for i, s in enumerate([(a * d, h), (k * d, h), (k * d, h), (h, a * d)])]
    U = dev(synth.normal_bf16((v, h), 0.3, 70))
    pages = -(-total // page)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(71)).int().reshape(1, pages).cuda()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    empty = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")

    class Model:
        def __init__(self):
            self.K, self.V = (torch.zeros(pages, k, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))

        def step(self, ids, length):
            """Settled tokens behind ids[0], which stands at position `length`, and the lead of the last one's logit."""
            M = len(ids)
            plan = tp.Plan(tp.make_config(tokens=M, hidden=h, n_heads=a, n_kv_heads=k, head_dim=d, tp_degree=t))
            n = tp.tp_plan_workspace_bytes(plan, tp.TP_OP_ATTN_CACHED)
            ws = torch.empty(n, dtype=torch.uint8, device="cuda")
            x, y, logits = empty(M, h), empty(M, h), empty(M, v)
            cache = tp.make_kv_cache(self.K, self.V, table, i32(0, M), i32(length + M), max_new=M)
            tp.tp_vocab_embedding_forward(i32(*ids), M, E, v, h, t, x)
            tp.tp_attn_cached_forward(plan, cache, x, *W, x, None, y, ws, n)
            tp.tp_vocab_logits_forward(y, M, h, U, v, t, logits)
            acc, tok = i32(0), torch.zeros(M, dtype=torch.int32, device="cuda")
            tp.tp_vocab_verify_drafts(logits, None, M, v, t, i32(*ids), i32(0, M), 1, torch.zeros(1, device="cuda"),
                                      torch.zeros(M, device="cuda"), None, acc, tok)
            sync_ok(plan)
            taken = int(acc)
            top = logits[taken].float().topk(2).values
            return tok.tolist()[:taken + 1], float(top[0] - top[1])

    plain, text, sure = Model(), [17], [True]
    while len(text) < total:
        got, lead = plain.step(text[-1:], len(text) - 1)
        text += got
        sure.append(lead > 0.5)             # a bf16 step of a logit near 16 is 2^-3, and the hidden state's steps add about as much
    fast, rng, at, steps, taken = Model(), np.random.default_rng(3), 1, 0, 0
    while at + 5 < total:
        right = int(rng.integers(0, 5))
        drafts, wrong = text[at:at + right], (text[at + right] + 1) % v
        got, _ = fast.step([text[at - 1]] + drafts + [wrong], at - 1)
        same = 0
        while same < len(got) and got[same] == text[at + same]:
            same += 1
        if same < len(got):
            assert not sure[at + same]
        if all(sure[at:at + right + 1]):
            assert got == text[at:at + right + 1]
            steps, taken = steps + 1, taken + right
        at += max(min(same, right + 1), 1)
    assert steps >= 5 and taken >= 5
