"""GPU parity of the operators of a training step around the blocks -- layer norm,
embedding, loss, output projection's gradients, clipping -- with their 64-bit
forms, through the C ABI.

Tolerances count roundings: a bf16 output is off by half a step, 2^-8 of the
value; fp32 sums of n terms by n 2^-24 of the sum of their magnitudes.  Where a
sum's order has fewer sequential steps than terms, the steps are counted."""
import ctypes as C

import numpy as np
import pytest
import torch

import megatron_tensor_transformer_colwise_gb300 as tp
import training_refs as refs
from gpu_util import assert_close, dev, host64

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8
U = 2.0 ** -24
EPS = 1e-5


def normal(shape, seed, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


def empty(*shape, dtype=torch.float32):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def scratch(n):
    return torch.full((max(n, 16),), 0xA5, dtype=torch.uint8, device="cuda")


def within(got, ref, bound, what):
    got = np.asarray(got, dtype=np.float64)
    if not got.size:
        return
    assert np.isfinite(got).all(), f"{what}: non-finite"
    over = np.abs(got - ref) - bound
    at = np.unravel_index(np.argmax(over), over.shape)
    assert over[at] <= 0, f"{what}{at}: {got[at]} for {ref[at]}, {over[at]:.3e} beyond its bound"


# ------------------------------------------------------------ layer norm

NORM_SIZES = [(1, 8), (1, 1024), (3, 256), (17, 264), (5, 512), (33, 520), (9, 1024), (4, 1032), (7, 2048), (6, 2056), (3, 2568),
              (5, 4096), (3, 4104), (2, 8192), (2, 8200), (3, 16384), (1000, 64), (2500, 768)]


def norm_inputs(rows, h, seed):
    x = normal((rows, h), seed, 1.0, torch.float32) * (torch.rand(rows, 1, generator=torch.Generator().manual_seed(seed)) * 3 + 0.01)
    x = (x + normal((rows, 1), seed + 1, 2.0, torch.float32)).bfloat16()
    return x, (1 + normal((h,), seed + 2, 0.3, torch.float32)).bfloat16(), normal((h,), seed + 3, 0.3), normal((rows, h), seed + 4), normal((rows, h), seed + 5)


def norm_bounds(x, eps=EPS):
    """Errors of the fp32 mean (48 steps of a sum: 32 in a thread, 5 shuffles, 16 warps, less where rows are short) and of
    1 / sqrt(variance + eps), relative (half of the variance's, plus the mean's error in every difference, plus the root's)."""
    n = 64
    mean, rstd = refs.layernorm_stats(x, eps)
    dmean = n * U * np.abs(x).mean(1)
    return mean, rstd, dmean, n * U + 0.5 * (dmean * rstd) ** 2 + np.abs(mean) * 2 * U * rstd


@pytest.mark.parametrize("rows,h", NORM_SIZES)
@pytest.mark.parametrize("affine", [True, False])
def test_layernorm_forward(rows, h, affine):
    x, gain, bias, _, _ = norm_inputs(rows, h, rows + h)
    y, stats = empty(rows, h, dtype=torch.bfloat16), empty(2, rows)
    g, b = (dev(gain), dev(bias)) if affine else (None, None)
    tp.tp_layernorm_forward(dev(x), rows, h, g, b, EPS, y, stats)
    X = host64(x)
    G, B = (host64(gain), host64(bias)) if affine else (1.0, 0.0)
    ref = refs.layernorm(X, G, B, EPS)
    mean, rstd, dmean, drstd = norm_bounds(X)
    inner = np.abs((X - mean[:, None]) * rstd[:, None] * G) * (drstd + 4 * U)[:, None] + (dmean * rstd)[:, None] * np.abs(G) + 2 * U * np.abs(ref)
    within(host64(y), ref, BF16 * np.abs(ref) + (1 + BF16) * inner, "y")
    st = host64(stats)
    within(st[0], mean, dmean, "mean")
    within(st[1], rstd, drstd * rstd, "rstd")
    again = empty(rows, h, dtype=torch.bfloat16)
    tp.tp_layernorm_forward(dev(x), rows, h, g, b, EPS, again)  # without statistics, the same bits
    inplace = dev(x).clone()
    tp.tp_layernorm_forward(inplace, rows, h, g, b, EPS, inplace)
    assert torch.equal(again, y) and torch.equal(inplace, y)


def run_norm_backward(x, gain, dy, dres, stats, rows, h, dgain=None, dbias=None, accumulate=False, dx=None):
    dx = empty(rows, h, dtype=torch.bfloat16) if dx is None else dx
    dgain = empty(h) if dgain is None else dgain
    dbias = empty(h) if dbias is None else dbias
    n = tp.tp_layernorm_backward_workspace_bytes(rows, h)
    tp.tp_layernorm_backward(x, rows, h, gain, EPS, stats, dy, dres, dx, dgain, dbias, accumulate, scratch(n), n)
    return dx, dgain, dbias


@pytest.mark.parametrize("rows,h", NORM_SIZES)
@pytest.mark.parametrize("kind", ["saved", "found", "residual", "plain"])
def test_layernorm_backward(rows, h, kind):
    x, gain, bias, dy, dres = norm_inputs(rows, h, 7 * rows + h)
    X, D = host64(x), host64(dy)
    G = 1.0 if kind == "plain" else host64(gain)
    R = host64(dres) if kind == "residual" else 0.0
    stats = None
    if kind in ("saved", "residual"):
        stats = empty(2, rows)
        tp.tp_layernorm_forward(dev(x), rows, h, None, None, EPS, empty(rows, h, dtype=torch.bfloat16), stats)
    g = None if kind == "plain" else dev(gain)
    r = dev(dres) if kind == "residual" else None
    dx, dgain, dbias = run_norm_backward(dev(x), g, dev(dy), r, stats, rows, h)
    rx, rg, rb, terms, sg, sb = refs.layernorm_backward(X, G, EPS, D, R)
    mean, rstd, dmean, drstd = norm_bounds(X)
    # xh is off by dmean rstd + drstd |xh|; every term of dx has two such factors, and sums of 64 steps.
    off = (dmean * rstd + 2 * drstd + 64 * U)[:, None]
    gabs = np.abs(D * G) * np.ones(h)
    spread = (rstd * dmean * rstd)[:, None] * (np.abs(((D * G) * (X - mean[:, None]) * rstd[:, None]).mean(1, keepdims=True)) + gabs.mean(1, keepdims=True) * np.abs((X - mean[:, None]) * rstd[:, None]))
    within(host64(dx), rx, BF16 * np.abs(rx) + (1 + BF16) * (4 * off * terms + 4 * spread), "dx")
    # Weights' sums: at most ceil(rows / CTAs) + 16 + 64 / 8 + 8 steps, held to 128 here, and xh's own error.
    within(host64(dgain), rg, 128 * U * sg + (off * np.abs(D) * (1 + np.abs((X - mean[:, None]) * rstd[:, None]))).sum(0), "dgain")
    within(host64(dbias), rb, 128 * U * sb, "dbias")
    again = run_norm_backward(dev(x), g, dev(dy), r, stats, rows, h)
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, dgain, dbias)))
    # In place of dy or of the residual's gradient; added to what is there; one of the two alone.
    d = dev(dy).clone()
    assert torch.equal(run_norm_backward(dev(x), g, d, r, stats, rows, h, dx=d)[0], dx)
    if r is not None:
        d = r.clone()
        assert torch.equal(run_norm_backward(dev(x), g, dev(dy), d, stats, rows, h, dx=d)[0], dx)
    old = normal((h,), 5, 1.0, torch.float32)
    more = run_norm_backward(dev(x), g, dev(dy), r, stats, rows, h, dgain=dev(old), dbias=dev(old), accumulate=True)
    assert torch.equal(more[1], dev(old) + dgain) and torch.equal(more[2], dev(old) + dbias)
    n = tp.tp_layernorm_backward_workspace_bytes(rows, h)
    only = empty(h)
    tp.tp_layernorm_backward(dev(x), rows, h, g, EPS, stats, dev(dy), r, dx, None, only, False, scratch(n), n)
    assert torch.equal(only, dbias)
    tp.tp_layernorm_backward(dev(x), rows, h, g, EPS, stats, dev(dy), r, dx, only, None, False, scratch(n), n)
    assert torch.equal(only, dgain)
    tp.tp_layernorm_backward(dev(x), rows, h, g, EPS, stats, dev(dy), r, again[0], None, None, False, None, 0)
    assert torch.equal(again[0], dx)


# Every shape of a row's warps, rows that fill it and rows that do not, more rows than the CTAs hold at a time.
@pytest.mark.parametrize("rows,h", [(3, 1536), (2, 1400), (2, 6144), (3, 6000), (2, 12288), (3, 10248), (5000, 520), (3100, 1032), (2500, 1536),
                                    (2100, 2568), (1500, 4096), (1300, 5000), (1000, 8192), (400, 12288)])
def test_layernorm_of_many_rows(rows, h):
    x, gain, bias, dy, dres = (dev(a) for a in norm_inputs(rows, h, rows + 3 * h))
    y, stats = empty(rows, h, dtype=torch.bfloat16), empty(2, rows)
    tp.tp_layernorm_forward(x, rows, h, gain, bias, EPS, y, stats)
    # The formulas in 64 bits on the GPU, tolerances as above.
    X, G, B, D, R = (a.double() for a in (x, gain, bias, dy, dres))
    mean = X.mean(1, keepdim=True)
    rstd = 1 / ((X - mean).square().mean(1, keepdim=True) + EPS).sqrt()
    xh = (X - mean) * rstd
    ref = xh * G + B
    dmean = 64 * U * X.abs().mean(1, keepdim=True)
    drstd = 64 * U + 0.5 * (dmean * rstd) ** 2 + mean.abs() * 2 * U * rstd
    inner = (xh * G).abs() * (drstd + 4 * U) + dmean * rstd * G.abs() + 2 * U * ref.abs()
    assert ((y.double() - ref).abs() <= BF16 * ref.abs() + (1 + BF16) * inner).all()
    assert ((stats[0].double() - mean[:, 0]).abs() <= dmean[:, 0]).all() and ((stats[1].double() / rstd[:, 0] - 1).abs() <= drstd[:, 0]).all()
    g = D * G
    gx = (g * xh).mean(1, keepdim=True)
    rx = R + rstd * (g - g.mean(1, keepdim=True) - xh * gx)
    terms = R.abs() + rstd * (g.abs() + g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    off = dmean * rstd + 2 * drstd + 64 * U
    spread = rstd * dmean * rstd * (gx.abs() + g.abs().mean(1, keepdim=True) * xh.abs())
    for st in (None, stats):
        dx, dgain, dbias = run_norm_backward(x, gain, dy, dres, st, rows, h)
        assert ((dx.double() - rx).abs() <= BF16 * rx.abs() + (1 + BF16) * (4 * off * terms + 4 * spread)).all()
        assert ((dgain.double() - (D * xh).sum(0)).abs() <= 128 * U * (D * xh).abs().sum(0) + (off * D.abs() * (1 + xh.abs())).sum(0)).all()
        assert ((dbias.double() - D.sum(0)).abs() <= 128 * U * D.abs().sum(0)).all()
        same = run_norm_backward(x, gain, dy, dres, st, rows, h)
        assert all(torch.equal(a, b) for a, b in zip(same, (dx, dgain, dbias)))
    inplace = x.clone()
    tp.tp_layernorm_forward(inplace, rows, h, gain, bias, EPS, inplace)
    assert torch.equal(inplace, y)


def test_layernorm_without_rows():
    g, b = dev(torch.ones(64)), dev(torch.ones(64))
    n = tp.tp_layernorm_backward_workspace_bytes(0, 64)
    for keep in (True, False):
        tp.tp_layernorm_backward(None, 0, 64, None, EPS, None, None, None, None, g, b, keep, scratch(n), n)
        assert float(g.sum()) == float(b.sum()) == (64.0 if keep else 0.0)


def test_layernorm_large_means_and_constant_rows():
    # A mean 200 times the spread, values of 2^55, and rows of one value (variance 0: y = bias).
    x = (200 + normal((4, 1024), 3, 1.0, torch.float32)).bfloat16()
    x[1] = (normal((1024,), 4, 1.0, torch.float32) * 2.0 ** 55).bfloat16()
    x[2] = 3.0
    x[3] = 0.0
    y, stats = empty(4, 1024, dtype=torch.bfloat16), empty(2, 4)
    tp.tp_layernorm_forward(dev(x), 4, 1024, None, None, EPS, y, stats)
    X = host64(x)
    ref = refs.layernorm(X, 1.0, 0.0, EPS)
    _, rstd, dmean, drstd = norm_bounds(X)
    within(host64(y), ref, BF16 * np.abs(ref) + 1.01 * (np.abs(ref) * (drstd + 8 * U)[:, None] + (dmean * rstd)[:, None]), "y")
    assert not host64(y)[2:].any()


def test_layernorm_keeps_nan_and_infinities_to_their_rows():
    x, gain, bias, dy, _ = norm_inputs(6, 640, 11)
    clean = empty(6, 640, dtype=torch.bfloat16)
    tp.tp_layernorm_forward(dev(x), 6, 640, dev(gain), dev(bias), EPS, clean)
    dclean = run_norm_backward(dev(x), dev(gain), dev(dy), None, None, 6, 640)[0]
    x[1, 5], x[3, 600] = float("nan"), float("inf")
    y = empty(6, 640, dtype=torch.bfloat16)
    tp.tp_layernorm_forward(dev(x), 6, 640, dev(gain), dev(bias), EPS, y)
    dx = run_norm_backward(dev(x), dev(gain), dev(dy), None, None, 6, 640)[0]
    for r in (0, 2, 4, 5):
        assert torch.equal(y[r], clean[r]) and torch.equal(dx[r], dclean[r])
    assert y[1].isnan().all() and y[3].isnan().any() and dx[1].isnan().all() and dx[3].isnan().any()


def test_layernorm_beyond_32_bit_offsets():
    rows, h = 140000, 16384
    x = torch.empty(rows, h, dtype=torch.bfloat16, device="cuda")
    x.random_(-3, 4)
    y = torch.empty_like(x)
    tp.tp_layernorm_forward(x, rows, h, None, None, EPS, y)
    at = [0, 131071, 131072, rows - 1]
    ref = refs.layernorm(host64(x[at]), 1.0, 0.0, EPS)
    within(host64(y[at]), ref, BF16 * np.abs(ref) + 2.0 ** -17 * (1 + np.abs(ref)), "y")
    dx, _, dbias = run_norm_backward(x, None, y, None, None, rows, h)
    rx, terms = (refs.layernorm_backward(host64(x[at]), 1.0, EPS, host64(y[at]))[i] for i in (0, 3))
    within(host64(dx[at]), rx, BF16 * np.abs(rx) + 2.0 ** -15 * terms, "dx")


# ------------------------------------------------------------ embedding

@pytest.mark.parametrize("M,v,h,t,scale", [(300, 4608, 128, 8, 11.3137085), (37, 512, 64, 1, 8.0), (1, 8, 8, 1, 0.3), (1000, 2048, 264, 4, -2.5)])
def test_embedding_scaled(M, v, h, t, scale):
    ids = torch.randint(0, v, (M,), generator=torch.Generator().manual_seed(M), dtype=torch.int32)
    if M > 10:
        ids[5], ids[6], ids[7], ids[8] = -3, v, 2 ** 31 - 1, -2 ** 31
    E = normal((v, h), 21)
    out = empty(M, h, dtype=torch.bfloat16)
    tp.tp_vocab_embedding_scaled_forward(dev(ids), M, dev(E), v, h, t, scale, out)
    ref = refs.embedding(ids.numpy(), host64(E), scale)
    within(host64(out), ref, BF16 * (1 + 2.0 ** -14) * np.abs(ref), "out")
    # A power of two is exact, and 1 is the plain lookup.
    plain = empty(M, h, dtype=torch.bfloat16)
    tp.tp_vocab_embedding_forward(dev(ids), M, dev(E), v, h, t, plain)
    tp.tp_vocab_embedding_scaled_forward(dev(ids), M, dev(E), v, h, t, 1.0, out)
    assert torch.equal(out, plain)
    tp.tp_vocab_embedding_scaled_forward(dev(ids), M, dev(E), v, h, t, 4.0, out)
    assert torch.equal(out, plain * 4)
    # Rows that no shard owns are zeros whatever the scale.
    tp.tp_vocab_embedding_scaled_forward(dev(ids), M, dev(E), v, h, t, float("inf"), out)
    if M > 10:
        assert not out[5:9].any()


def words(M, v, kind, seed):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, v, (M,), generator=g, dtype=torch.int32)
    if kind == "one":
        ids[:] = v - 1
    elif kind == "few":
        ids = ids % min(v, 3)
    elif kind == "text":
        ids = (v * torch.rand(M, generator=g) ** 6).to(torch.int32).clamp(max=v - 1)
    elif kind == "strange":
        ids[::5], ids[1::7], ids[2::11] = -1, v, 2 ** 31 - 1
        ids[3::13] = -2 ** 31
    elif kind == "ends":
        ids[: M // 2], ids[M // 2 :] = 0, v - 1
    elif kind == "none":
        ids[:] = -100
    return ids


def run_embedding_backward(ids, v, dOut, scale, dE=None, accumulate=False, t=1):
    M, h = dOut.shape
    dE = empty(v, h) if dE is None else dE
    n = tp.tp_vocab_embedding_backward_workspace_bytes(M, v, h)
    tp.tp_vocab_embedding_backward(ids, M, v, h, t, scale, dOut, dE, accumulate, scratch(n), n)
    return dE


@pytest.mark.parametrize("M,v,h,t", [(1, 8, 8, 1), (31, 8, 16, 2), (33, 1000, 40, 4), (300, 4608, 128, 8), (1023, 257, 264, 1),
                                     (5000, 2056, 72, 1), (64, 32768, 1024, 4), (700, 31, 1032, 1), (129, 1, 4104, 1), (2050, 512, 8, 8)])
@pytest.mark.parametrize("kind", ["any", "one", "few", "text", "strange", "ends", "none"])
def test_embedding_backward(M, v, h, t, kind):
    ids, dOut, scale = words(M, v, kind, M + v), normal((M, h), M + h), 1.7
    dE = run_embedding_backward(dev(ids), v, dev(dOut), scale, t=t)
    ref, size, count = refs.embedding_backward(ids.numpy(), v, host64(dOut), scale)
    within(host64(dE), ref, (count[:, None] + 2) * U * size, "dE")
    assert torch.equal(run_embedding_backward(dev(ids), v, dev(dOut), scale, t=t), dE)
    # Added to what is there; words without a token keep their bits, NaN among them.
    old = normal((v, h), 5, 1.0, torch.float32)
    unseen = torch.from_numpy(count == 0)
    old[unseen] = float("nan")
    got = run_embedding_backward(dev(ids), v, dev(dOut), scale, dev(old), True, t)
    assert torch.equal(got.cpu().view(torch.int32)[unseen], old.view(torch.int32)[unseen])
    seen = count > 0
    with np.errstate(invalid="ignore"):
        want = host64(old) + ref
    if seen.any():
        within(host64(got)[seen], want[seen], (count[:, None] + 3)[seen] * U * (size + np.abs(host64(old)))[seen], "dE added")


def test_embedding_backward_without_tokens():
    n = tp.tp_vocab_embedding_backward_workspace_bytes(0, 40, 16)
    dE = dev(torch.ones(40, 16))
    tp.tp_vocab_embedding_backward(None, 0, 40, 16, 2, 1.0, None, dE, True, scratch(n), n)
    assert float(dE.sum()) == 640
    tp.tp_vocab_embedding_backward(None, 0, 40, 16, 2, 1.0, None, dE, False, scratch(n), n)
    assert not dE.any()


def test_embedding_beyond_32_bit_offsets():
    v, h = 131080, 16392
    ids = torch.tensor([0, v - 1, 131009, v - 1], dtype=torch.int32)
    dOut = normal((4, h), 77)
    dE = torch.full((v, h), 3.0, device="cuda")
    run_embedding_backward(dev(ids), v, dev(dOut), 1.0, dE)
    ref, size, count = refs.embedding_backward(np.array([0, 2, 1, 2]), 3, host64(dOut), 1.0)
    within(host64(dE[[0, 131009, v - 1]]), ref, 3 * U * size, "dE")
    assert not dE[1:131009].any() and not dE[131010 : v - 1].any()
    E = dE.bfloat16()
    out = empty(4, h, dtype=torch.bfloat16)
    tp.tp_vocab_embedding_scaled_forward(dev(ids), 4, E, v, h, 1, 2.0, out)
    assert torch.equal(out, 2 * E[ids.long()])


@pytest.mark.parametrize("M,v,h", [(70001, 3000, 64), (700001, 40, 8), (9000, 70000, 1032)])
def test_embedding_backward_of_many_tokens(M, v, h):
    # More tokens than a word's part holds, half of them one word: against torch's sums in 64 bits.
    ids, dOut = words(M, v, "text", 9), normal((M, h), 10)
    ids[::2] = 1717 % v
    dE = run_embedding_backward(dev(ids), v, dev(dOut), 1.0)
    at = dev(ids).long()
    ref = torch.zeros(v, h, dtype=torch.float64, device="cuda").index_add_(0, at, dev(dOut).double())
    size = torch.zeros(v, h, dtype=torch.float64, device="cuda").index_add_(0, at, dev(dOut).double().abs())
    count = torch.bincount(at, minlength=v)[:, None]
    assert ((dE.double() - ref).abs() <= (count + 2) * U * size).all()


# ------------------------------------------------------------ loss

def run_loss(logits, labels, dloss, t=1, out=None):
    M, v = logits.shape
    loss, d = empty(M), empty(M, v, dtype=torch.bfloat16) if out is None else out
    tp.tp_vocab_parallel_cross_entropy_train(logits, M, v, t, labels, dloss, loss, d)
    return loss, d


def loss_close(z, labels, dloss, loss, d):
    """dlogits: probabilities off by 2^-14 (a sum of up to 300 steps in fp32, exponents off by 100 2^-24) and one rounding;
    those below 2^-126 count as 0.  loss: the same relative error, whose label's share does not come from a difference."""
    Z = host64(z)
    with np.errstate(all="ignore"):
        rl, rd = refs.loss(Z, labels.numpy(), dloss)
    gl, gd = host64(loss), host64(d)
    np.testing.assert_array_equal(np.isnan(gl), np.isnan(rl))
    np.testing.assert_array_equal(np.isinf(gl), np.isinf(rl))
    np.testing.assert_array_equal(np.isnan(gd), np.isnan(rd))
    f = np.isfinite(rl)
    within(gl[f], rl[f], 2.0 ** -14 * np.abs(rl[f]) + 2.0 ** -126, "loss")
    f = np.isfinite(rd)
    bound = (BF16 + 2.0 ** -13) * np.abs(rd) + 2.0 ** -125 * (1 + np.abs(np.asarray(dloss)))[:, None]
    assert (np.abs(gd - rd)[f] <= bound[f]).all(), float((np.abs(gd - rd) - bound)[f].max())


@pytest.mark.parametrize("M,v,t", [(1, 8, 1), (5, 64, 8), (3, 4096, 4), (7, 4104, 1), (129, 1024, 1), (300, 4608, 8), (3, 32768, 4),
                                   (2, 50264, 1), (2, 128256, 8), (1, 262152, 1), (37, 264, 1)])
@pytest.mark.parametrize("scale", [1.0, 8.0])
def test_loss_and_gradient(M, v, t, scale):
    z = normal((M, v), M + v, scale)
    labels = torch.randint(0, v, (M,), generator=torch.Generator().manual_seed(v), dtype=torch.int32)
    labels[0] = v - 1
    if M > 2:
        labels[1], labels[2] = -100, 0
    if M > 4:
        labels[3], labels[4] = v, -1
    w = torch.rand(M, generator=torch.Generator().manual_seed(1)) + 0.1
    loss, d = run_loss(dev(z), dev(labels), dev(w), t)
    loss_close(z, labels, w.double().numpy(), loss, d)
    if M > 2:
        assert float(loss[1]) == 0 and not d[1].any()
    # dloss of 1, the logits' own buffer, and the plain loss's answer.
    ones, d1 = run_loss(dev(z), dev(labels), None, t)
    loss_close(z, labels, np.ones(M), ones, d1)
    own = dev(z).clone()
    same, d2 = run_loss(own, dev(labels), dev(w), t, out=own)
    assert torch.equal(d2.view(torch.int16), d.view(torch.int16)) and torch.equal(same.view(torch.int32), loss.view(torch.int32))
    plain, stats = empty(M), empty(3 * t * M)
    tp.tp_vocab_parallel_cross_entropy(dev(z), M, v, t, dev(labels), stats, plain)
    ok = ~plain.isnan().cpu()
    assert torch.equal(ok, ~loss.isnan().cpu())
    assert ((plain - loss).cpu()[ok].abs() <= 2.0 ** -14 * loss.cpu()[ok].abs() + 2.0 ** -18).all()


def test_loss_of_masked_logits():
    v = 4104
    z = normal((9, v), 3, 2.0)
    labels = torch.full((9,), 17, dtype=torch.int32)
    z[0, 2000:] = -np.inf                      # padding words
    z[1, :] = -np.inf
    z[1, 17] = 1.5                             # the label alone: loss 0, no gradient
    z[2, 17] = -np.inf                         # the label is masked: infinite loss, finite gradient
    z[3, :] = -np.inf                          # nothing: NaN
    z[4, 100] = float("nan")
    z[5, 100] = np.inf
    z[6, :] = torch.finfo(torch.bfloat16).min  # the type's lowest value everywhere: uniform
    z[7, 1:] = torch.finfo(torch.bfloat16).min
    z[7, 0] = torch.finfo(torch.bfloat16).max
    labels[8] = -100
    z[8, :] = float("nan")                     # an ignored row counts for nothing, whatever it holds
    w = torch.ones(9)
    w[8] = float("nan")
    loss, d = run_loss(dev(z), dev(labels), dev(w))
    w[8] = 1.0
    loss_close(z, labels, w.double().numpy(), loss, d)
    assert float(loss[1]) == 0 and not d[1].any() and float(loss[8]) == 0 and not d[8].any()
    assert float(loss[2]) == np.inf and d[3].isnan().all() and d[4].isnan().all() and d[5].isnan().all()


@pytest.mark.parametrize("M,v", [(6000, 520), (1500, 16384), (700, 20000), (400, 50264), (160, 128256), (80, 200000)])
def test_loss_of_many_rows(M, v):
    # More rows than the clusters hold at a time, ignored and wrong labels among them, in runs and alone.
    z = normal((M, v), M, 3.0)
    g = torch.Generator().manual_seed(v)
    labels = torch.randint(0, v, (M,), generator=g, dtype=torch.int32)
    labels[torch.rand(M, generator=g) < 0.3] = -100
    labels[M // 3 : M // 3 + M // 5] = -100
    labels[torch.rand(M, generator=g) < 0.02] = v
    labels[-1] = -100
    w = torch.rand(M, generator=g)
    loss, d = run_loss(dev(z), dev(labels), dev(w))
    loss_close(z, labels, w.double().numpy(), loss, d)
    # The same bits in place, captured and replayed, and beside another call on another stream.
    own, other = dev(z).clone(), dev(z).clone()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    lab, up = dev(labels), dev(w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run_loss(own, lab, up, out=own)[0]
    assert torch.equal(own, dev(z))
    torch.cuda.synchronize()
    for stream, call in ((a, graph.replay), (b, lambda: run_loss(other, lab, up, out=other))):
        with torch.cuda.stream(stream):
            call()
    torch.cuda.synchronize()
    for x in (own, other):
        assert torch.equal(x.view(torch.int16), d.view(torch.int16))
    assert torch.equal(held.view(torch.int32), loss.view(torch.int32))


@pytest.mark.parametrize("t", [1, 3])
def test_plain_loss_of_masked_words(t):
    # tp_vocab_parallel_cross_entropy: words that a thread or a shard sees alone may all be masked.
    M, v = 6, 4104
    z = normal((M, v), 8, 2.0)
    z[0, 1368:] = -np.inf
    z[1, :2736] = -np.inf
    z[2, :] = -np.inf
    z[2, 17] = 1.5
    z[3, 8:] = -np.inf
    z[4, :] = -np.inf
    z[5, :] = -np.inf
    z[5, 2000] = np.nan
    labels = torch.tensor([17, 4000, 17, 3, 17, 17], dtype=torch.int32)
    loss, stats = empty(M), empty(3 * t * M)
    tp.tp_vocab_parallel_cross_entropy(dev(z), M, v, t, dev(labels), stats, loss)
    ref = refs.loss(host64(z), labels.numpy(), np.ones(M))[0]
    got = host64(loss)
    assert np.isnan(got[4:]).all()
    # exponents off by 2^-24 of up to 16, a logarithm and a difference of numbers up to 16.
    within(got[:4], ref[:4], 2.0 ** -18 * (1 + np.abs(ref[:4])), "loss")


def test_loss_small_ones_and_far_logits():
    # The label far ahead of all others: 1 - p would vanish in fp32.
    v = 1000
    z = torch.zeros(4, v, dtype=torch.bfloat16)
    for r, lead in enumerate((20.0, 30.0, 60.0, -90.0)):
        z[r, 3] = lead
    labels = torch.full((4,), 3, dtype=torch.int32)
    loss, d = run_loss(dev(z), dev(labels), None)
    loss_close(z, labels, np.ones(4), loss, d)
    assert float(loss[1]) > 0 and float(d[1, 3]) < 0
    z = normal((3, v), 4, 1.0, torch.float32) + torch.tensor([[3.0e4], [-3.0e4], [1e30]])
    loss, d = run_loss(dev(z.bfloat16()), dev(labels[:3]), None)
    loss_close(z.bfloat16(), labels[:3], np.ones(3), loss, d)


def test_loss_gradient_against_differences():
    v, e = 520, 2.0 ** -4
    z = (torch.randint(-12, 13, (40, v), generator=torch.Generator().manual_seed(8)) / 8).bfloat16()
    z[:] = z[0]
    z[0::4, 7] += 3
    labels = torch.full((40,), 7, dtype=torch.int32)
    up, down = z.clone(), z.clone()
    at = torch.arange(40) * 13 % v
    at[0::4] = 7
    row = torch.arange(40)
    up[row, at] += e
    down[row, at] -= e
    d = run_loss(dev(z), dev(labels), None)[1].float().cpu()[row, at]
    diff = (run_loss(dev(up), dev(labels), None)[0] - run_loss(dev(down), dev(labels), None)[0]).cpu() / (2 * e)
    # Third derivative at most 1/8 here (p (1-p) (1-2p) and the like): e^2 / 6 / 8; fp32 losses off by 2^-20.
    assert ((d - diff).abs() <= e * e / 48 + 2.0 ** -19 / e + BF16 * d.abs()).all()


def test_loss_beyond_32_bit_offsets():
    M, v = 17000, 128256
    z = torch.empty(M, v, dtype=torch.bfloat16, device="cuda")
    z.random_(-4, 5)
    labels = torch.randint(0, v, (M,), dtype=torch.int32, device="cuda")
    at = torch.tensor([0, 16743, 16744, M - 1], device="cuda")
    keep = z[at].clone()
    loss, d = run_loss(z, labels, None, out=z)
    loss_close(keep.cpu(), labels[at].cpu(), np.ones(4), loss[at], d[at])


def test_loss_without_tokens():
    tp.tp_vocab_parallel_cross_entropy_train(None, 0, 64, 4, None, None, None, None)
    torch.cuda.synchronize()


# ------------------------------------------------------------ output projection's gradients

def run_output(H, W, d, dH=None, dW=None, accumulate=False, t=1, want=(True, True)):
    (M, h), v = H.shape, W.shape[0]
    dH = (empty(M, h, dtype=torch.bfloat16) if dH is None else dH) if want[0] else None
    dW = (empty(v, h) if dW is None else dW) if want[1] else None
    n = tp.tp_vocab_logits_backward_workspace_bytes(M, v, h)
    tp.tp_vocab_logits_backward(H, M, h, W, v, t, d, dH, dW, accumulate, scratch(n) if n else None, n)
    return dH, dW


SEG = 768  # tokens of dW that one tensor-core sum takes


@pytest.mark.parametrize("M,v,h,t", [(1, 8, 8, 1), (5, 64, 16, 8), (130, 2048, 64, 2), (300, 4608, 128, 8), (257, 1032, 264, 1), (64, 32768, 256, 4),
                                     (700, 8200, 520, 1), (1024, 50264, 72, 1)])
def test_output_gradients(M, v, h, t):
    H, W, d = normal((M, h), 1), normal((v, h), 2), normal((M, v), 3)
    dH, dW = run_output(dev(H), dev(W), dev(d), t=t)
    D, Hd, Wd = dev(d).double(), dev(H).double(), dev(W).double()
    # A sum of n products in the tensor cores: n / 16 steps, each off by at most 2^-22 of the running magnitude.
    rh = D @ Wd
    within(host64(dH), rh.cpu().numpy(), (BF16 * rh.abs() + (v / 16 + 16) * 2.0 ** -22 * (D.abs() @ Wd.abs())).cpu().numpy(), "dH")
    rw, sw = D.T @ Hd, D.abs().T @ Hd.abs()
    within(host64(dW), rw.cpu().numpy(), ((M / 16 + 16) * 2.0 ** -22 * sw).cpu().numpy(), "dW")
    one = run_output(dev(H), dev(W), dev(d), t=t, want=(True, False))[0]
    two = run_output(dev(H), dev(W), dev(d), t=t, want=(False, True))[1]
    assert torch.equal(one, dH) and torch.equal(two, dW)
    old = normal((v, h), 4, 1.0, torch.float32)
    more = run_output(dev(H), dev(W), dev(d), dW=dev(old).clone(), accumulate=True, t=t)[1]
    # Sums s1, s2, .. of SEG tokens each, the same bits in both calls, are added in order:
    # each partial sum old + s1 + .. + sj is rounded once, and without old each but s1 itself,
    # so that the two differ by at most U (sum over j of |old + s1 + .. + sj| + sum over j > 1
    # of |s1 + .. + sj|).  The partial sums are taken from 64 bits; what the tensor cores'
    # fall short of those, below 2^-20 of the sum of magnitudes here, counts beside them.
    old64, bound = host64(old), U * np.abs(host64(old) + host64(dW))
    for at in range(SEG, M, SEG):
        s = (D[:at].T @ Hd[:at]).cpu().numpy()
        bound = bound + U * (1 + 2.0 ** -10) * np.abs(old64 + s) + U * 2.0 ** -20 * (np.abs(old64) + sw.cpu().numpy())
    if M > SEG:
        parts = [np.abs((D[:at].T @ Hd[:at]).cpu().numpy()) for at in range(2 * SEG, M, SEG)] + [np.abs(host64(dW))]
        bound = bound + U * (1 + 2.0 ** -10) * sum(parts)
    within(host64(more), old64 + host64(dW), bound, "dW added")


@pytest.mark.parametrize("M,v,h", [(2500, 520, 264), (4100, 1032, 128), (1025, 264, 520)])
def test_output_gradients_of_many_tokens(M, v, h):
    # Several sums of SEG tokens each, added to what is there, the same bits every time.
    H, W, d, old = normal((M, h), 1), normal((v, h), 2), normal((M, v), 3), normal((v, h), 4, 30.0, torch.float32)
    x = [dev(a) for a in (H, W, d)]
    dW = run_output(*x)[1]
    D, Hd = x[2].double(), x[0].double()
    ref, size = D.T @ Hd, D.abs().T @ Hd.abs()
    bound = (SEG / 16 + 16) * 2.0 ** -22 * size + (M / SEG + 1) * U * (size + dev(old).double().abs())
    assert ((dW.double() - ref).abs() <= bound).all()
    more = run_output(*x, dW=dev(old).clone(), accumulate=True)[1]
    assert ((more.double() - ref - dev(old).double()).abs() <= bound).all()
    for _ in range(5):
        assert torch.equal(run_output(*x)[1], dW) and torch.equal(run_output(*x, dW=dev(old).clone(), accumulate=True)[1], more)
    # Whole numbers: exact, whatever the segments.
    Hi, di = ((torch.randint(-3, 4, a.shape, generator=torch.Generator().manual_seed(5))).bfloat16() for a in (H, d))
    assert torch.equal(run_output(dev(Hi), x[1], dev(di))[1].double(), dev(di).double().T @ dev(Hi).double())


def test_output_gradients_integers_bit_exact():
    M, v, h = 300, 4616, 128
    g = torch.Generator().manual_seed(3)
    H, W, d = (torch.randint(-2, 3, s, generator=g).bfloat16() for s in ((M, h), (v, h), (M, v)))
    d[:, 50:] *= (torch.rand(M, v - 50, generator=g) < 0.02)  # sums that bf16 holds
    dH, dW = run_output(dev(H), dev(W), dev(d))
    rh, rw = d.double() @ W.double(), d.double().T @ H.double()
    assert torch.equal(dH.cpu(), rh.bfloat16()) and torch.equal(dW.cpu().double(), rw)


def test_output_gradients_without_tokens():
    dW = dev(torch.ones(64, 16))
    tp.tp_vocab_logits_backward(None, 0, 16, dev(torch.zeros(64, 16).bfloat16()), 64, 2, None, None, dW, True, None, 0)
    assert float(dW.sum()) == 1024
    tp.tp_vocab_logits_backward(None, 0, 16, dev(torch.zeros(64, 16).bfloat16()), 64, 2, None, None, dW, False, None, 0)
    assert not dW.any()


# ------------------------------------------------------------ clipping

def run_clip(grads, max_norm, out="new"):
    dst = [torch.full_like(g, float("nan")) for g in grads] if out == "new" else out
    items = tp.make_grad_list(grads, dst)
    norm = empty(1)
    n = tp.tp_grad_clip_workspace_bytes(len(items))
    tp.tp_grad_clip(items, max_norm, norm, scratch(n), n)
    return float(norm), dst if dst is not None else grads


def clip_close(grads, max_norm, norm, out):
    """Squares are summed a few dozen at a time in fp32 (64 steps at most, halved by the root), the rest in fp64."""
    rn, ro = refs.clip([host64(g).reshape(-1) for g in grads], max_norm)
    assert abs(norm - rn) <= 2.0 ** -18 * rn + 2.0 ** -149, (norm, rn)
    for g, o, r in zip(grads, out, ro):
        half = U if g.dtype == torch.float32 else BF16
        least = 2.0 ** -149 if g.dtype == torch.float32 else 2.0 ** -133
        within(host64(o).reshape(-1), r, (half + 2.0 ** -17) * np.abs(r) + least, "clipped")


CLIP_SIZES = [[1], [7, 8, 9], [8191], [8192], [8193, 1, 0, 16385], [1000003, 5, 262144], list(range(1, 60)), [3] * 700, [100] * 33]


@pytest.mark.parametrize("sizes", CLIP_SIZES, ids=lambda s: f"{len(s)}x{sum(s)}")
@pytest.mark.parametrize("ratio", [0.5, 1.5, 30.0])
def test_clip(sizes, ratio):
    grads = [dev(normal((n,), 3 + i, 0.1 * (i % 4 + 1), torch.bfloat16 if i % 3 == 1 else torch.float32)) for i, n in enumerate(sizes)]
    max_norm = refs.clip([host64(g) for g in grads], 1.0)[0] / ratio
    keep = [g.clone() for g in grads]
    norm, out = run_clip(grads, max_norm)
    clip_close(grads, max_norm, norm, out)
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))
    if ratio < 1:
        assert all(torch.equal(a, b) for a, b in zip(out, grads))
    assert run_clip(grads, max_norm)[0] == norm
    there = [None if i % 2 else torch.zeros_like(g) for i, g in enumerate(grads)]  # some only measured
    assert run_clip(grads, max_norm, there)[0] == norm
    assert all(b is None or torch.equal(a, b) for a, b in zip(out, there))
    same, own = run_clip(grads, max_norm, None)  # in place
    assert same == norm and all(torch.equal(a, b) for a, b in zip(own, out))


@pytest.mark.parametrize("value", [1e30, 3e38, 1e-25, 1e-38, 1e-44, 0.0])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_clip_neither_overflows_nor_vanishes(value, dtype):
    n = 20001
    g = torch.zeros(n, dtype=dtype)
    g[::3] = value
    g[5] = -value
    r = float(np.sqrt((host64(g) ** 2).sum()))
    for max_norm in (r / 3, r * 2, 1e-30):
        max_norm = float(np.float32(min(max_norm, 3e38)))
        norm, out = run_clip([dev(g), dev(torch.zeros(100))], max_norm)
        if r > 3.4e38:
            assert norm == np.inf  # above fp32, and clipped all the same
            norm = r
        clip_close([g, torch.zeros(100)], max_norm, norm, out)


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_clip_tells_of_infinities_and_nan(bad):
    g = [dev(normal((9000,), 1, 1.0, torch.float32)), dev(normal((77,), 2))]
    g[1][70] = bad
    norm, out = run_clip(g, 0.5)
    assert not np.isfinite(norm) and np.isnan(norm) == np.isnan(bad)
    for a, b in zip(g, out):
        np.testing.assert_array_equal(host64(a), host64(b))


def test_clip_limits():
    g = [dev(normal((500,), 1, 1.0, torch.float32))]
    norm, out = run_clip(g, float("inf"))
    assert torch.equal(out[0], g[0]) and norm > 0
    assert not run_clip(g, 0.0)[1][0].any()
    n = tp.tp_grad_clip_workspace_bytes(0)
    norm = empty(1)
    tp.tp_grad_clip(tp.make_grad_list([]), 1.0, norm, scratch(n), n)
    assert float(norm) == 0
    assert run_clip([torch.empty(0, device="cuda")], 1.0)[0] == 0


def test_clip_beyond_32_bit_offsets():
    n = (1 << 31) + 8200
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    at = [0, (1 << 31) - 1, 1 << 31, n - 1]
    g[at] = torch.tensor([3.0, 4.0, 12.0, 84.0], device="cuda").bfloat16()
    norm, out = run_clip([g], 8.5, None)
    assert norm == 85.0  # 3, 4, 12, 84: all sums and the root are whole numbers
    assert out[0][at].float().tolist() == [float(torch.tensor(x * 8.5 / norm).bfloat16()) for x in (3.0, 4.0, 12.0, 84.0)]


# ------------------------------------------------------------ together

class Step:
    """A training step of a small model around the GeLU MLP: scaled embedding, norm, MLP with its residual, norm, output
    projection with the embedding's weights, mean loss; backward; clipping."""

    M, h, f, v, t = 96, 128, 256, 520, 1

    def __init__(self, seed):
        M, h, f, v = self.M, self.h, self.f, self.v
        self.E, self.W1, self.W2 = normal((v, h), seed, 0.05), normal((f, h), seed + 1, 0.08), normal((h, f), seed + 2, 0.08)
        self.g1, self.b1 = (1 + normal((h,), seed + 3, 0.1, torch.float32)).bfloat16(), normal((h,), seed + 4, 0.1)
        self.g2, self.b2 = (1 + normal((h,), seed + 5, 0.1, torch.float32)).bfloat16(), normal((h,), seed + 6, 0.1)
        g = torch.Generator().manual_seed(seed + 7)
        self.ids = (v * torch.rand(M, generator=g) ** 3).to(torch.int32)
        self.labels = torch.randint(0, v, (M,), generator=g, dtype=torch.int32)
        self.labels[::9] = -100
        live = int((self.labels != -100).sum())
        self.dloss = torch.full((M,), 1.0 / live)
        self.scale = float(np.sqrt(h))
        self.max_norm = 0.25

    def on_gpu(self):
        M, h, f, v, t = self.M, self.h, self.f, self.v, self.t
        s = {n: dev(getattr(self, n)) for n in ("E", "W1", "W2", "g1", "b1", "g2", "b2", "ids", "labels", "dloss")}
        bf = lambda *shape: empty(*shape, dtype=torch.bfloat16)
        s.update(x=bf(M, h), xn=bf(M, h), y=bf(M, h), yn=bf(M, h), UG=bf(M, f), logits=bf(M, v), loss=empty(M), st1=empty(2, M), st2=empty(2, M),
                 dyn=bf(M, h), dy=bf(M, h), dxn=bf(M, h), dx=bf(M, h), norm=empty(1))
        s["grads"] = {n: empty(*s[n].shape) for n in ("E", "W1", "W2", "g1", "b1", "g2", "b2")}
        s["plan"] = tp.Plan(tp.make_config(tokens=M, hidden=h, ffn=f, tp_degree=2, act="gelu"))
        s["list"] = tp.make_grad_list(s["grads"].values())
        n = max(tp.tp_plan_workspace_bytes(s["plan"], tp.TP_OP_MLP), tp.tp_plan_workspace_bytes(s["plan"], tp.TP_OP_MLP_BACKWARD),
                tp.tp_layernorm_backward_workspace_bytes(M, h), tp.tp_vocab_embedding_backward_workspace_bytes(M, v, h),
                tp.tp_vocab_logits_backward_workspace_bytes(M, v, h), tp.tp_grad_clip_workspace_bytes(7))
        s["ws"], s["n"] = scratch(n), n
        return s

    def run(self, s):
        M, h, v, t = self.M, self.h, self.v, self.t
        g, ws, n = s["grads"], s["ws"], s["n"]
        tp.tp_vocab_embedding_scaled_forward(s["ids"], M, s["E"], v, h, t, self.scale, s["x"])
        tp.tp_layernorm_forward(s["x"], M, h, s["g1"], s["b1"], EPS, s["xn"], s["st1"])
        tp.tp_mlp_forward_train(s["plan"], s["xn"], s["W1"], None, s["W2"], None, s["x"], None, s["y"], s["UG"], ws, n)
        tp.tp_layernorm_forward(s["y"], M, h, s["g2"], s["b2"], EPS, s["yn"], s["st2"])
        tp.tp_vocab_logits_forward(s["yn"], M, h, s["E"], v, t, s["logits"])
        tp.tp_vocab_parallel_cross_entropy_train(s["logits"], M, v, t, s["labels"], s["dloss"], s["loss"], s["logits"])
        tp.tp_vocab_logits_backward(s["yn"], M, h, s["E"], v, t, s["logits"], s["dyn"], g["E"], False, ws, n)
        tp.tp_layernorm_backward(s["y"], M, h, s["g2"], EPS, s["st2"], s["dyn"], None, s["dy"], g["g2"], g["b2"], False, ws, n)
        tp.tp_mlp_backward(s["plan"], s["xn"], s["W1"], None, s["W2"], s["dy"], s["UG"], s["dxn"], g["W1"], None, g["W2"], None, False, ws, n)
        tp.tp_layernorm_backward(s["x"], M, h, s["g1"], EPS, s["st1"], s["dxn"], s["dy"], s["dx"], g["g1"], g["b1"], False, ws, n)
        tp.tp_vocab_embedding_backward(s["ids"], M, v, h, t, self.scale, s["dx"], g["E"], True, ws, n)
        tp.tp_grad_clip(s["list"], self.max_norm, s["norm"], ws, n)
        return s["loss"], s["norm"], *g.values()

    def reference(self):
        p = {n: getattr(self, n).double().requires_grad_() for n in ("E", "W1", "W2", "g1", "b1", "g2", "b2")}
        F = torch.nn.functional
        x = self.scale * p["E"][self.ids.long()]
        y = x + F.gelu(F.layer_norm(x, (self.h,), p["g1"], p["b1"], EPS) @ p["W1"].T) @ p["W2"].T
        z = F.layer_norm(y, (self.h,), p["g2"], p["b2"], EPS) @ p["E"].T
        loss = F.cross_entropy(z, self.labels.long(), reduction="none", ignore_index=-100)
        (loss * self.dloss.double()).sum().backward()
        norm, grads = refs.clip([p[n].grad.numpy() for n in p], self.max_norm)
        return [loss.detach().numpy(), np.array([norm]), *grads]


def test_training_step_against_autograd():
    step = Step(500)
    got = step.run(step.on_gpu())
    for a, b, n in zip(got, step.reference(), ("loss", "norm", "E", "W1", "W2", "g1", "b1", "g2", "b2")):
        assert_close(host64(a), b, what=n)


def test_training_step_captured_and_replayed():
    steps = [Step(600), Step(700)]
    eager = [[x.clone() for x in s.run(s.on_gpu())] for s in steps]
    states = [s.on_gpu() for s in steps]
    for s, st in zip(steps, states):
        s.run(st)
    torch.cuda.synchronize()
    # One graph each with its own workspace, replayed side by side on two streams; then the second one's inputs in the first.
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in steps]
    for s, st in zip(steps, states):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(s.run(st))
        graphs.append(g)
    for o in outs:
        for x in o:
            x.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(20):
        for g, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                g.replay()
    torch.cuda.synchronize()
    for o, e in zip(outs, eager):
        assert all(torch.equal(a, b) for a, b in zip(o, e))
    for n in ("E", "W1", "W2", "g1", "b1", "g2", "b2", "ids", "labels", "dloss"):
        states[0][n].copy_(states[1][n])
    graphs[0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs[0], eager[1]))


def test_training_operators_on_other_streams():
    steps = [Step(800 + 10 * i) for i in range(3)]
    eager = [[x.clone() for x in s.run(s.on_gpu())] for s in steps]
    states = [s.on_gpu() for s in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(5):
        outs = []
        for s, st, stream in zip(steps, states, streams):
            with torch.cuda.stream(stream):
                outs.append(s.run(st))
    torch.cuda.synchronize()
    for o, e in zip(outs, eager):
        assert all(torch.equal(a, b) for a, b in zip(o, e))
