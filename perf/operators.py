"""Cases of the serving operators: the paged key/value cache (write, quantising
or not, and read back), attention of new tokens over that cache, and the
verification of drafted tokens against the target's probabilities.

``run`` computes an operator in its plain form, in elementary torch operations,
or, where ``own`` is true, calls the package's entry point for it.

Shapes (a query heads, k key/value heads of dimension d, t shards):
QKV is the shard-blocked projection buffer [M][t * W], W = (a/t + 2 kv) d with
kv = max(k/t, 1) key/value heads a shard; the cache is [pages][k][page][d], with
[pages][k][page] fp32 scales where it holds 8-bit values; sequence s owns the
rows q_start[s] .. q_start[s+1] of QKV, its new tokens, which stand at the
positions kv_len[s] - (their number) .. kv_len[s] - 1 of its page-table row.
"""
import itertools
import math
import random

import torch

own = False

E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100  # the least magnitude that a row's 448 stands for
AMAX_CEIL = 3.3895313892515355e38  # the largest finite bf16


# ------------------------------------------------------------ cases

def _cache(name, op, heads, kv_heads, head_dim, tp, kv, page, seqs, ctx_lo, ctx_hi, new_lo, new_hi, chunks=0, chunk=0,
           lens=1, pad=0):
    return {"name": name, "op": op, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "tp": tp, "kv": kv,
            "page": page, "seqs": seqs, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "new_lo": new_lo, "new_hi": new_hi,
            "chunks": chunks, "chunk": chunk, "lens": lens, "pad": pad}


def _verify(name, seqs, drafts_lo, drafts_hi, vocab, tp, greedy, lens=1, pad=0):
    return {"name": name, "op": "verify", "seqs": seqs, "drafts_lo": drafts_lo, "drafts_hi": drafts_hi, "vocab": vocab,
            "tp": tp, "greedy": greedy, "lens": lens, "pad": pad}


def listed():
    return [
        # One decoding step of a batch: each sequence appends its one new token.
        _cache("write 64x1 bf16", "write", 32, 8, 128, 8, "bf16", 64, 64, 200, 4000, 1, 1, lens=11),
        # The prompts of four sequences enter an 8-bit cache at once.
        _cache("write 4x2048 e4m3", "write", 32, 8, 128, 8, "e4m3", 64, 4, 0, 0, 2048, 2048, lens=12),
        # A few short sequences taken out of the cache, small heads, small pages, replicated key/value heads.
        _cache("read 8 short bf16", "read", 16, 2, 64, 4, "bf16", 16, 8, 30, 1000, 1, 1, lens=13),
        # Long sequences brought back from 8 bits, as for moving them elsewhere.
        _cache("read 16 long e4m3", "read", 32, 8, 128, 8, "e4m3", 64, 16, 2000, 16000, 1, 1, lens=14),
        # One user, one token: the latency of the smallest call.
        _cache("attend 1x1 over 4k bf16", "attend", 32, 8, 128, 8, "bf16", 64, 1, 4096, 4096, 1, 1, lens=15),
        # Decoding of a ragged batch.
        _cache("attend 64x1 ragged bf16", "attend", 32, 8, 128, 8, "bf16", 64, 64, 500, 16000, 1, 1, lens=16),
        # The same from an 8-bit cache, which holds longer contexts.
        _cache("attend 64x1 ragged e4m3", "attend", 32, 8, 128, 8, "e4m3", 128, 64, 1000, 32000, 1, 1, lens=17),
        # Drafted tokens of each sequence, eight query heads a key/value head, replicated shards, small pages.
        _cache("attend 32x(2..6) drafted d64", "attend", 16, 2, 64, 8, "bf16", 16, 32, 300, 8000, 2, 6, lens=18, pad=7),
        # A long prompt's next chunk: bound by arithmetic.
        _cache("attend 2048 over 8k bf16", "attend", 32, 8, 128, 8, "bf16", 64, 1, 8192, 8192, 2048, 2048, lens=19),
        # Chunks of prompts and single tokens in one call, from 8 bits.
        _cache("attend mixed e4m3", "attend", 32, 8, 128, 4, "e4m3", 32, 24, 300, 6000, 1, 1, chunks=3, chunk=500, lens=20),
        # Drafts of two sequences.
        _verify("verify 2x(3+1) 32k", 2, 3, 3, 32768, 4, 0, lens=21),
        # Drafts of a whole batch, every eighth sequence greedy.
        _verify("verify 64x(2..5+1) 128k", 64, 2, 5, 128256, 8, 8, lens=22, pad=3),
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["write", "read", "attend", "attend", "attend", "verify"])
        lens = rng.randrange(1 << 20)
        if op == "verify":
            hi = rng.randint(1, 6)
            c = _verify("", _log_between(rng, 1, 80), rng.randint(0, hi), hi, 8 * _log_between(rng, 100, 16032), 1,
                        rng.choice([0, 1, 2, 5]), lens, rng.choice([0, 0, 5]))
        else:
            kv_heads = rng.choice([1, 2, 4, 8])
            group = rng.choice([1, 2, 3, 4, 6, 8])
            tp = rng.choice([t for t in (1, 2, 4, 8) if (kv_heads * group) % t == 0 and
                             (kv_heads % t == 0 or t % kv_heads == 0)])
            ctx_hi = _log_between(rng, 20, 32000)
            ctx_lo = rng.randint(1, ctx_hi)
            kind = rng.choice(["decode", "drafted", "chunk", "mixed"])
            new_hi = {"decode": 1, "drafted": rng.randint(2, 9), "chunk": _log_between(rng, 10, 2048), "mixed": 1}[kind]
            chunks, chunk = (rng.randint(1, 3), _log_between(rng, 10, 700)) if kind == "mixed" else (0, 0)
            seqs = _log_between(rng, 1, 64 if kind in ("decode", "drafted") else 8) + chunks
            c = _cache("", op, kv_heads * group, kv_heads, rng.choice([64, 128]), tp, rng.choice(["bf16", "e4m3"]),
                       rng.choice([16, 32, 64, 128]), seqs, ctx_lo, ctx_hi, max(1, new_hi - rng.randint(0, new_hi)),
                       new_hi, chunks, chunk, lens, rng.choice([0, 0, 3]))
        del c["name"]
        if _cost(c) <= 170e-6 and _plain_floats(c) <= 6e9:
            return c


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.8e15)


def _plain_floats(case):
    """Scores that the plain form holds at a time."""
    if case["op"] == "verify":
        return case["seqs"] * (case["drafts_hi"] + 1) * case["vocab"]
    new, kv = _lengths(case)
    return len(new) * case["heads"] * max(new) * max(kv)


def _lengths(case):
    """New tokens and whole length of each sequence: of the case alone."""
    rng = random.Random(case["lens"])
    n = case["seqs"]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(n)]
    for i in rng.sample(range(n), min(n, case["chunks"])):
        new[i] = case["chunk"]
    ctx = [_log_between(rng, case["ctx_lo"], case["ctx_hi"]) if case["ctx_hi"] > 0 else 0 for _ in range(n)]
    return new, [x + y for x, y in zip(new, ctx)]


def _drafts(case):
    rng = random.Random(case["lens"])
    return [rng.randint(case["drafts_lo"], case["drafts_hi"]) + 1 for _ in range(case["seqs"])]


def work(case):
    if case["op"] == "verify":
        rows = sum(_drafts(case))
        logits = (2 * rows - case["seqs"]) * case["vocab"]  # no draft distribution at a sequence's last row
        return {"bytes": 2.0 * logits + 4.0 * case["seqs"] * case["vocab"] + 16 * rows,
                "flops": 4.0 * logits + 4.0 * case["seqs"] * case["vocab"]}
    new, kv = _lengths(case)
    a, k, d = case["heads"], case["kv_heads"], case["head_dim"]
    elem, scales = (2, 0) if case["kv"] == "bf16" else (1, 8)
    if case["op"] == "write":
        n = float(sum(new)) * k
        return {"bytes": n * (2 * d * (2 + elem) + scales), "flops": n * 4 * d}
    if case["op"] == "read":
        n = float(sum(kv)) * k
        return {"bytes": n * (2 * d * (2 + elem) + scales), "flops": n * 2 * d}
    seen = sum(n * (l - n) + n * (n + 1) // 2 for n, l in zip(new, kv))  # keys that each new token sees
    return {"bytes": float(sum(kv)) * k * (2 * d * elem + scales) + 4.0 * sum(new) * a * d, "flops": 4.0 * seen * a * d}


# ------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, g, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(lens):
    return [0, *itertools.accumulate(lens)]


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "verify":
        return _prepare_verify(case, g)
    new, kv = _lengths(case)
    a, k, d, t, page = (case[x] for x in ("heads", "kv_heads", "head_dim", "tp", "page"))
    width = (a // t + 2 * max(k // t, 1)) * d
    rows = sum(new) + case["pad"]
    need = [-(-n // page) for n in kv]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    column = torch.arange(max(need), device="cuda")
    first = _ints(_starts(need))[:-1]
    table = torch.where(column < _ints(need)[:, None], order[(first[:, None] + column).clamp(max=pages - 1)], -1)
    st = {"case": dict(case), "QKV": _normal((rows, t * width), g), "table": table.to(torch.int32).contiguous(),
          "q_start": _ints(_starts(new)), "kv_len": _ints(kv), "tokens": sum(new), "max_new": max(new),
          "max_len": max(kv), "k_scale": None, "v_scale": None}
    if case["kv"] == "bf16":
        st["K"], st["V"] = (_normal((pages, k, page, d), g) for _ in range(2))
    else:
        st["K"], st["V"] = (_normal((pages, k, page, d), g).mul_(80).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn) for _ in range(2))
        st["k_scale"], st["v_scale"] = (torch.rand((pages, k, page), generator=g, device="cuda") * 0.02 + 0.004
                                        for _ in range(2))
    if case["op"] == "read":
        st["K_out"], st["V_out"] = (torch.zeros((len(kv), max(kv), k, d), dtype=torch.bfloat16, device="cuda")
                                    for _ in range(2))
    if case["op"] == "attend":
        st["O"] = _normal((rows, a * d), g)
    if own:
        import megatron_tensor_transformer_colwise_gb300 as tp
        st["plan"] = tp.Plan(tp.make_config(tokens=rows, hidden=a * d, n_heads=a, n_kv_heads=k, head_dim=d, tp_degree=t))
        st["cache"] = tp.make_kv_cache(st["K"], st["V"], st["table"], st["q_start"], st["kv_len"], st["k_scale"],
                                       st["v_scale"], max_new=st["max_new"])
        if case["op"] == "attend":
            st["ws_bytes"] = tp.tp_plan_workspace_bytes(st["plan"], tp.TP_OP_ATTN_PAGED)
            st["ws"] = torch.empty(st["ws_bytes"], dtype=torch.uint8, device="cuda")
    return st


def _prepare_verify(case, g):
    rows = _drafts(case)
    n, M, v = len(rows), sum(rows) + case["pad"], case["vocab"]
    # A draft model that is near the target: about three drafts in four are taken.
    logits = _normal((M, v), g).mul_(2.5)
    draft = (logits + _normal((M, v), g).mul_(0.6)).to(torch.bfloat16)
    temperature = torch.rand(n, generator=g, device="cuda") * 0.6 + 0.6
    if case["greedy"]:
        temperature[:: case["greedy"]] = 0.0
    at = _starts(rows)
    seq = torch.repeat_interleave(torch.arange(n, device="cuda"), _ints(rows))
    scale = torch.where(temperature > 0, 1 / temperature.clamp(min=1e-3), 50.0)[seq]
    race = torch.rand((at[-1], v), generator=g, device="cuda").clamp_(min=1e-9).log_().neg_().log_().neg_()
    drawn = (draft[: at[-1]].float() * scale[:, None]).add_(race).argmax(1).to(torch.int32)
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    ids[1 : at[-1]] = drawn[:-1]
    return {"case": dict(case), "logits": logits, "draft": draft, "ids": ids, "q_start": _ints(at), "temperature": temperature,
            "u": torch.rand(M, generator=g, device="cuda"), "noise": torch.empty((n, v), device="cuda").exponential_(generator=g),
            "accepted": torch.zeros(n, dtype=torch.int32, device="cuda"), "rows": at[-1], "most": max(rows),
            "out": torch.zeros(M, dtype=torch.int32, device="cuda")}


# ------------------------------------------------------------ the operators

def run(state):
    return {"write": _write, "read": _read, "attend": _attend, "verify": _verify_drafts}[state["case"]["op"]](state)


def _rows(st):
    """Of each new token: its sequence, its number in it, and its position."""
    start = st["q_start"].long()
    row = torch.arange(st["tokens"], device="cuda")
    seq = torch.searchsorted(start, row, right=True) - 1
    nth = row - start[seq]
    return seq, nth, st["kv_len"][seq] - (start[1:] - start[:-1])[seq] + nth


def _heads(st, part):
    """Q [M][a][d], or K or V [M][k][d], out of the projection buffer."""
    c = st["case"]
    a, k, d, t = c["heads"], c["kv_heads"], c["head_dim"], c["tp"]
    kv = max(k // t, 1)
    x = st["QKV"][: st["tokens"]].view(st["tokens"], t, a // t + 2 * kv, d)
    if part == "Q":
        return x[:, :, : a // t].reshape(-1, a, d)
    x = x[:, :, a // t : a // t + kv] if part == "K" else x[:, :, a // t + kv :]
    return (x if k >= t else x[:, :: t // k]).reshape(-1, k, d)


def _written(st):
    return {n: st[n] for n in ("K", "V", "k_scale", "v_scale") if st[n] is not None}


def _write(st):
    if own:
        import megatron_tensor_transformer_colwise_gb300 as tp
        tp.tp_kv_cache_write(st["plan"], st["cache"], st["QKV"])
        return _written(st)
    page = st["case"]["page"]
    seq, _, pos = _rows(st)
    at, off = st["table"][seq, pos // page].long(), pos % page
    _put(st, "K", "k_scale", at, off)
    _put(st, "V", "v_scale", at, off)
    return _written(st)


def _put(st, part, scale, at, off):
    x = _heads(st, part)
    if st[scale] is None:
        st[part][at, :, off] = x
        return
    x = x.float()
    amax = x.abs().amax(2).clamp(AMAX_FLOOR, AMAX_CEIL)
    st[scale][at, :, off] = amax / E4M3_MAX
    back = torch.full_like(amax, E4M3_MAX) / amax  # one rounding: a number over a tensor is a reciprocal's multiple
    x = (x * back[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    st[part].view(torch.uint8)[at, :, off] = x.view(torch.uint8)


def _gathered(st, part, scale):
    """[sequences][padded length][k][d] in 32 bits, from the pages."""
    x = st[part][st["table"].clamp(min=0).long()].float()
    if st[scale] is not None:
        x = x * st[scale][st["table"].clamp(min=0).long()][..., None]
    s, p, k, n, d = x.shape
    return x.transpose(2, 3).reshape(s, p * n, k, d)[:, : st["max_len"]]


def _read(st):
    if own:
        import megatron_tensor_transformer_colwise_gb300 as tp
        tp.tp_kv_cache_read(st["plan"], st["cache"], st["max_len"], st["K_out"], st["V_out"])
        return [st["K_out"], st["V_out"]]
    live = (torch.arange(st["max_len"], device="cuda") < st["kv_len"][:, None])[:, :, None, None]
    st["K_out"].copy_(torch.where(live, _gathered(st, "K", "k_scale").to(torch.bfloat16), st["K_out"]))
    st["V_out"].copy_(torch.where(live, _gathered(st, "V", "v_scale").to(torch.bfloat16), st["V_out"]))
    return [st["K_out"], st["V_out"]]


def _attend(st):
    if own:
        import megatron_tensor_transformer_colwise_gb300 as tp
        tp.tp_attn_paged_forward(st["plan"], st["cache"], st["QKV"], st["O"], st["ws"], st["ws_bytes"])
        return st["O"]
    c = st["case"]
    k, d = c["kv_heads"], c["head_dim"]
    seq, nth, pos = _rows(st)
    n, most, group = len(st["kv_len"]), st["max_new"], c["heads"] // k
    q = torch.zeros((n, most, k, group, d), device="cuda")
    q[seq, nth] = _heads(st, "Q").float().view(-1, k, group, d)
    at = torch.full((n, most), -1, dtype=torch.long, device="cuda")
    at[seq, nth] = pos
    K = _gathered(st, "K", "k_scale").permute(0, 2, 3, 1)
    s = (q.permute(0, 2, 1, 3, 4).reshape(n, k, most * group, d) @ K).mul_(1 / math.sqrt(d))
    unseen = torch.arange(st["max_len"], device="cuda") > at.repeat_interleave(group, 1)[:, None, :, None]
    s = s.masked_fill_(unseen, -math.inf)
    p = (s - s.amax(3, keepdim=True).clamp(min=-1e30)).exp_()
    o = p @ _gathered(st, "V", "v_scale").permute(0, 2, 1, 3) / p.sum(3, keepdim=True).clamp(min=1e-30)
    o = o.view(n, k, most, group, d).transpose(1, 2)[seq, nth]
    st["O"][: st["tokens"]] = o.reshape(st["tokens"], -1).to(torch.bfloat16)
    return st["O"]


def _first_largest(x):
    """The lowest index of the largest value of each row."""
    n = x.shape[-1]
    return torch.where(x == x.amax(-1, keepdim=True), torch.arange(n, device="cuda"), n).amin(-1)


def _verify_drafts(st):
    c = st["case"]
    if own:
        import megatron_tensor_transformer_colwise_gb300 as tp
        tp.tp_vocab_verify_drafts(st["logits"], st["draft"], st["logits"].shape[0], c["vocab"], c["tp"], st["ids"],
                                  st["q_start"], c["seqs"], st["temperature"], st["u"], st["noise"], st["accepted"], st["out"])
        return [st["accepted"], st["out"]]
    # Padded to the longest sequence: probabilities in 64 bits, since a decision is next to a border now and then.
    start = st["q_start"].long()
    number = start[1:] - start[:-1]
    nth = torch.arange(st["most"], device="cuda")
    row = (start[:-1, None] + nth).clamp(max=st["rows"] - 1)
    greedy = st["temperature"] <= 0
    heat = torch.where(greedy, 1.0, st["temperature"]).double()[:, None, None]
    z, y = st["logits"][row], st["draft"][row]
    p = (z.double() / heat).softmax(-1)
    q = (y.double() / heat).softmax(-1)
    top = _first_largest(z)
    x = st["ids"][(row + 1).clamp(max=st["rows"] - 1)].long()
    taken = st["u"][row].double() * q.gather(2, x[..., None])[..., 0] < p.gather(2, x[..., None])[..., 0]
    taken = torch.where(greedy[:, None], x == top, taken) & (nth < number[:, None] - 1)
    count = taken.int().cumprod(1).sum(1)
    last = count[:, None, None].expand(-1, 1, c["vocab"])
    p, q = p.gather(1, last)[:, 0], q.gather(1, last)[:, 0]
    left = torch.where((count < number - 1)[:, None], (p - q).clamp(min=0), p)
    left = torch.where(left.amax(1, keepdim=True) > 0, left, p)
    token = torch.where(greedy, top.gather(1, count[:, None])[:, 0], _first_largest(left / st["noise"].double()))
    out = torch.where(nth < count[:, None], x, torch.where(nth == count[:, None], token[:, None], -1)).to(torch.int32)
    seq = torch.searchsorted(start, torch.arange(st["rows"], device="cuda"), right=True) - 1
    st["out"][: st["rows"]] = out[seq, torch.arange(st["rows"], device="cuda") - start[seq]]
    st["accepted"].copy_(count)
    return [st["accepted"], st["out"]]


# ------------------------------------------------------------ the definitions in 64 bits

def _to_e4m3(y):
    """The nearest value with a sign, 3 bits of fraction and exponents -6 .. 8 (ties to even, at most 448)."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -60))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def exact(case, seed):
    if case["op"] == "verify":
        return None  # whole numbers alone
    st = prepare(case, seed)
    new, kv = _lengths(case)
    a, k, d, t, page = (case[x] for x in ("heads", "kv_heads", "head_dim", "tp", "page"))
    apart = (a // t + 2 * max(k // t, 1)) * d

    def column(part, head):
        if part == "Q":
            return head // (a // t) * apart + head % (a // t) * d
        shard, local = (head // (k // t), head % (k // t)) if k >= t else (head * (t // k), 0)
        return shard * apart + (a // t + local + (max(k // t, 1) if part == "V" else 0)) * d

    def cached(part, s, g):
        n = -(-kv[s] // page)
        at = st["table"][s, :n].long()
        x = st[part][at, g].double()
        scale = st["k_scale" if part == "K" else "v_scale"]
        return (x if scale is None else x * scale[at, g].double()[..., None]).reshape(n * page, d)[: kv[s]]

    if case["op"] == "write":
        out = {n: (x.float() if "K" in n or "V" in n else x).double() for n, x in _written(st).items()}
        first = 0
        for s, n in enumerate(new):
            pos = torch.arange(kv[s] - n, kv[s], device="cuda")
            at, off = st["table"][s, pos // page].long(), pos % page
            for g in range(k):
                for part, scale in (("K", "k_scale"), ("V", "v_scale")):
                    j = column(part, g)
                    x = st["QKV"][first : first + n, j : j + d].double()
                    if case["kv"] == "e4m3":
                        most = x.abs().amax(1).clamp(AMAX_FLOOR, AMAX_CEIL)
                        out[scale][at, g, off] = most / 448
                        x = _to_e4m3(x * (448 / most)[:, None])
                    out[part][at, g, off] = x
            first += n
        return out
    if case["op"] == "read":
        outs = []
        for part in ("K", "V"):
            out = st[part + "_out"].double()
            for s in range(len(kv)):
                for g in range(k):
                    out[s, : kv[s], g] = cached(part, s, g)
            outs.append(out)
        return outs
    out, first = st["O"].double(), 0
    for s, n in enumerate(new):
        hidden = torch.arange(kv[s], device="cuda") > torch.arange(kv[s] - n, kv[s], device="cuda")[:, None]
        for g in range(k):
            K, V = cached("K", s, g), cached("V", s, g)
            for j in range(g * (a // k), (g + 1) * (a // k)):
                i = column("Q", j)
                q = st["QKV"][first : first + n, i : i + d].double()
                p = torch.softmax((q @ K.T / d ** 0.5).masked_fill(hidden, -math.inf), 1)
                out[first : first + n, j * d : (j + 1) * d] = p @ V
        first += n
    return out
