"""Inputs and plain 64-bit forms of the serving operators (not a test module):
the paged key/value cache, attention over it, and draft verification.

A ``Paged`` problem holds everything on the host.  Whatever no sequence owns
is poison: cache rows past a sequence's length and unused pages hold NaN, so
an operator that lets them in shows it.
"""
import math

import numpy as np
import torch

import megatron_tensor_transformer_colwise_gb300 as tp

E4M3_NAN = 0x7F


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3 fraction bits."""
    c = np.arange(256)
    s = np.where(c & 0x80, -1.0, 1.0)
    e, f = (c >> 3) & 15, c & 7
    v = np.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * 2.0 ** (e - 7.0))
    return np.where((c & 0x7F) == E4M3_NAN, np.nan, s * v)


VALUES = e4m3_values()


def quantise(x: np.ndarray):
    """(codes, scales) of rows x [..., d] (float64 of bf16 values), by the header's definition: its
    three fp32 roundings, then the nearest code, ties to the even one, at most 448."""
    with np.errstate(all="ignore"):
        amax = np.fmax(np.fmax.reduce(np.abs(x), axis=-1), 2.0 ** -100)
        amax = np.minimum(amax, 3.3895313892515355e38).astype(np.float32)
        scale = amax / np.float32(448)
        y = (x.astype(np.float32) * (np.float32(448) / amax)[..., None]).astype(np.float64)
        a = np.minimum(np.abs(y), 448.0)
        e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6)
        step = 2.0 ** (e - 3)
        r = np.round(np.where(np.isnan(a), 0, a) / step) * step  # numpy rounds half to even
    code = np.searchsorted(VALUES[:E4M3_NAN], r)
    code = np.where(np.isnan(y), E4M3_NAN, code) | np.where(np.signbit(y), 0x80, 0)
    return code.astype(np.uint8), scale


class Paged:
    """lens: (new tokens, whole length) of each sequence."""

    def __init__(self, a, k, d, t, page, lens, kv="bf16", seed=0, pad=0, first=0, spare=2, scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.a, self.k, self.d, self.t, self.page, self.kv = a, k, d, t, page, kv
        self.new, self.len = [n for n, _ in lens], [m for _, m in lens]
        self.n_seqs = len(lens)
        self.held = max(k // t, 1)
        self.shard = (a // t + 2 * self.held) * d
        self.start = np.cumsum([first] + self.new)
        self.rows = int(self.start[-1]) + pad
        self.QKV = (torch.randn(self.rows, t * self.shard, generator=g) * scale).to(torch.bfloat16)
        need = [-(-m // page) for m in self.len]
        self.n_pages = sum(need) + spare
        order = torch.randperm(self.n_pages, generator=g).tolist()
        self.table = np.full((self.n_seqs, max(need + [1])), -1, dtype=np.int32)
        used = 0
        for s, n in enumerate(need):
            self.table[s, :n] = order[used:used + n]
            used += n
        shape = (self.n_pages, k, page, d)
        if kv == "bf16":
            self.K, self.V = (torch.full(shape, math.nan, dtype=torch.bfloat16) for _ in range(2))
            self.ks = self.vs = None
        else:
            self.K, self.V = (torch.full(shape, E4M3_NAN, dtype=torch.uint8) for _ in range(2))
            self.ks, self.vs = (torch.full(shape[:3], math.nan) for _ in range(2))
        for s in range(self.n_seqs):  # what earlier calls and this one's append left there
            for p in range(self.len[s]):
                pg, off = self.table[s, p // page], p % page
                if kv == "bf16":
                    self.K[pg, :, off] = (torch.randn(k, d, generator=g) * scale).to(torch.bfloat16)
                    self.V[pg, :, off] = (torch.randn(k, d, generator=g) * scale).to(torch.bfloat16)
                else:
                    for c, sc in ((self.K, self.ks), (self.V, self.vs)):
                        code = torch.randint(0, 254, (k, d), generator=g)
                        c[pg, :, off] = (code + (code >= E4M3_NAN)).to(torch.uint8)  # every code but the NaNs
                        sc[pg, :, off] = torch.rand(k, generator=g) * 0.01 * scale + 1e-4

    # ---- device side

    def config(self, **kw):
        return tp.make_config(tokens=self.rows, hidden=kw.pop("hidden", 64), n_heads=self.a, n_kv_heads=self.k,
                              head_dim=self.d, tp_degree=self.t, **kw)

    def upload(self, max_new=None):
        """(plan, cache) with the cache's tensors on the current device (cache.tensors keeps them)."""
        to = lambda x: None if x is None else x.cuda()
        i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()
        cache = tp.make_kv_cache(to(self.K), to(self.V), i32(self.table), i32(self.start), i32(self.len), to(self.ks),
                                 to(self.vs), max_new=max(self.new, default=0) if max_new is None else max_new)
        return tp.Plan(self.config()), cache

    # ---- plain forms, float64

    def column(self, part, head):
        """First column of query head `head`, or of KV head `head` where it is held first."""
        per = self.a // self.t
        if part == "Q":
            return head // per * self.shard + head % per * self.d
        shard, local = (head // self.held, head % self.held) if self.k >= self.t else (head * (self.t // self.k), 0)
        return shard * self.shard + (per + local + (self.held if part == "V" else 0)) * self.d

    def projected(self, part):
        """[rows][heads][d]"""
        x = self.QKV.double().numpy()
        n = self.a if part == "Q" else self.k
        return np.stack([x[:, self.column(part, h):self.column(part, h) + self.d] for h in range(n)], axis=1)

    def position(self, s, i):
        return self.len[s] - self.new[s] + i

    def written(self):
        """(K, V, k_scale, v_scale) after the append, as numpy arrays of what the cache stores."""
        out = []
        for part, c, sc in (("K", self.K, self.ks), ("V", self.V, self.vs)):
            x = self.projected(part)
            if self.kv == "bf16":
                c, sc = c.view(torch.int16).numpy().copy(), None
                x = self.bits(part)
            else:
                c, sc = c.numpy().copy(), sc.numpy().copy()
                x, scale = quantise(x)
            for s in range(self.n_seqs):
                for i in range(self.new[s]):
                    p = self.position(s, i)
                    if p < 0 or p >= self.page * self.table.shape[1]:
                        continue
                    pg = self.table[s, p // self.page]
                    if not 0 <= pg < self.n_pages:
                        continue
                    c[pg, :, p % self.page] = x[self.start[s] + i]
                    if sc is not None:
                        sc[pg, :, p % self.page] = scale[self.start[s] + i]
            out += [c, sc]
        return out[0], out[2], out[1], out[3]

    def bits(self, part):
        x = self.QKV.view(torch.int16).numpy()
        return np.stack([x[:, self.column(part, h):self.column(part, h) + self.d] for h in range(self.k)], axis=1)

    def cached(self, part, s):
        """[len][k][d] values of sequence s; zeros where the page is not one of the cache's."""
        c, sc = (self.K, self.ks) if part == "K" else (self.V, self.vs)
        out = np.zeros((self.len[s], self.k, self.d))
        for p in range(min(self.len[s], self.page * self.table.shape[1])):
            pg = self.table[s, p // self.page]
            if 0 <= pg < self.n_pages:
                x = c[pg, :, p % self.page]
                out[p] = x.double().numpy() if sc is None else \
                    VALUES[x.numpy()] * sc[pg, :, p % self.page].double().numpy()[:, None]
        return out

    def attention(self):
        """(O, A, E) [rows][a][d]: the outputs (zeros where no sequence owns the row or nothing is seen),
        sum p |v|, the size that roundings of the probabilities act on, and for an 8-bit cache
        max (p vs) sum |code|, the size that the smallest weights' absolute rounding acts on."""
        Q = self.projected("Q")
        O = np.zeros((self.rows, self.a, self.d))
        A, E = np.zeros_like(O), np.zeros_like(O)
        for s in range(self.n_seqs):
            K, V = self.cached("K", s), self.cached("V", s)
            vs = np.abs(V).max(axis=2, keepdims=True) / 448 + 1e-300  # at most the scale
            for i in range(self.new[s]):
                n = self.position(s, i) + 1
                if n <= 0:
                    continue
                r = self.start[s] + i
                for j in range(self.a):
                    g = j // (self.a // self.k)
                    x = K[:n, g] @ Q[r, j] / math.sqrt(self.d)
                    p = np.exp(x - x.max())
                    p /= p.sum()
                    O[r, j] = p @ V[:n, g]
                    A[r, j] = p @ np.abs(V[:n, g])
                    if self.kv != "bf16":
                        E[r, j] = (p * vs[:n, g, 0]).max() * (np.abs(V[:n, g]) / vs[:n, g]).sum(axis=0)
        return O, A, E

    def owned(self):
        m = np.zeros(self.rows, dtype=bool)
        m[self.start[0]:self.start[-1]] = True
        return m


def attention_tolerance(O, A, E):
    """Elementwise bound on a bf16 attention output's error.  Each probability is rounded to bf16 (half
    a step, 2^-8 of its value) before the product with V: at most 2^-8 A with A = sum p |v|.  The output
    is rounded to bf16 once: 2^-8 |O|.  A score is an fp32 sum of d exact products, off by at most
    (d + 2) 2^-24 sum |q k| / sqrt d <= 130 * 2^-24 * 12 < 2^-13 for standard normal Q and K at d <= 128
    (sum |q k| / sqrt d is about 7 there), which moves a probability by that share and the sum of
    probabilities by no more: 2^-12 A.  exp2's 2^-22 and fp32 accumulation stay below what that leaves.
    With 8-bit V the weights p vs are rounded to fp16 with the largest at 2^15: to 2^-11 of themselves, or
    by at most 2^-25, 2^-40 of the largest, where they fall below fp16's normal range; times the codes
    that is 2^-40 E (one power of two more for E's scales, which are at most the true ones)."""
    return 2.0 ** -8 * (A + np.abs(O)) + 2.0 ** -12 * A + 2.0 ** -39 * E


def softmax64(x, T):
    x = np.asarray(x, dtype=np.float64) / T
    m = x.max()
    if m == -math.inf:
        return np.zeros_like(x)
    e = np.exp(x - m)
    return e / e.sum()


def verify(logits, draft, ids, start, temperature, u, noise):
    """(accepted, tokens, margin): float64 by the header's definition; tokens is -2 in rows that no
    sequence owns.  margin[s] is the least relative distance of sequence s's decisions from their
    borders: where it is small an fp32 evaluation may rightly decide otherwise."""
    logits = np.asarray(logits, dtype=np.float64)
    M, v = logits.shape
    tokens = np.full(M, -2, dtype=np.int64)
    accepted = np.zeros(len(start) - 1, dtype=np.int64)
    margin = np.full(len(start) - 1, math.inf)
    for s in range(len(start) - 1):
        r0, n = int(start[s]), int(start[s + 1] - start[s])
        T = 1.0 if temperature is None else float(temperature[s])
        greedy = not T > 0
        tokens[r0:r0 + n] = -1
        for i in range(n):
            r, last = r0 + i, i + 1 == n
            x = -1 if last else int(ids[r + 1])
            inside = 0 <= x < v
            if greedy:
                token = int(np.argmax(logits[r])) if logits[r].max() > -math.inf else -1
                if not last and inside and x == token:
                    tokens[r] = x
                    accepted[s] += 1
                    continue
                tokens[r] = token
                break
            p = softmax64(logits[r], T)
            q = np.zeros(v) if last or draft is None else softmax64(np.asarray(draft[r], dtype=np.float64), T)
            if not last and inside:
                left, right = float(u[r]) * q[x], p[x]
                margin[s] = min(margin[s], abs(left - right) / max(left, right, 1e-300))
                if left < right:
                    tokens[r] = x
                    accepted[s] += 1
                    continue
            w = np.maximum(p - q, 0)
            if not w.max() > 0:
                w = p
            race = w / (np.ones(v) if noise is None else np.asarray(noise[s], dtype=np.float64))
            tokens[r] = int(np.argmax(race)) if race.max() > 0 else -1
            best = np.sort(race)[-2:]
            # p - q carries an error of (p + q) times that of one probability.
            k = tokens[r]
            grown = max(1.0, (p[k] + q[k]) / max(w[k], 1e-300)) if k >= 0 else 1.0
            if v > 1 and best[-1] > 0:
                margin[s] = min(margin[s], (best[-1] - best[-2]) / best[-1] / grown)
            break
    return accepted, tokens, margin
