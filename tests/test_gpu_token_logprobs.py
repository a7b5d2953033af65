"""Token log-probabilities and their gradient through gpt2k_token_logprobs and
gpt2k_token_logprobs_bwd, against numpy in 64 bits.

Tolerances, with eps = 2^-24 (half a step of fp32). z = x / tau has a relative error of
at most 3 eps (the reciprocal, the product, a difference), so d = z - m has an absolute
one of 6 eps Z with Z = max(|m|, |z|) over the row's entries that count (those within
e^-40 of the largest: the rest is below 1e-17 of the sum). The sum s of V positive terms:
each has that error plus exp's (2^-21), and the additions add at most eps for each of the
V / 128 + 16 additions in a row that a term can go through. So
  D(log s) = 6 eps Z + 2^-21 + (V / 128 + 16) eps,
log p = d - log s and lse = m + log s add a rounding of the result and the error of d,
and the entropy log s - w / s the same error again, weighted by |d| <= 40 in the worst
term: sum p |d| (2^-21 + ...) <= (H + 2) of it. Gradients: p = e^(z - lse) has the relative
error 6 eps (|z| + |lse|) + 2^-21, its factor g + h (log p + H) the absolute one
|h| (6 eps (|z| + |lse| + H)) + 3 eps of its parts; a bf16 result adds 2^-8. A p below the
smallest normal number, 2^-126, is flushed to zero (ex2.approx.ftz): it is off by less than 2^-126, and its product with
its factor by less than 2^-126 of that (with a factor of 100 that is 1.2e-36)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
KINDS = ["normal", "equal", "up", "down", "empty", "one_left", "lowest", "half_masked", "nan", "inf", "few_values",
         "peak", "signed_zeros", "few_left", "crowded", "ties"]


def _rows(kinds, V, dtype, seed):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((len(kinds), V)) * 3).astype(np.float32)
    low = float(torch.finfo(dtype).min)
    for r, kind in enumerate(kinds):
        if kind == "equal":
            x[r] = 1.5
        elif kind == "up":
            x[r] = np.linspace(-9, 9, V)
        elif kind == "down":
            x[r] = np.linspace(9, -9, V)
        elif kind == "empty":
            x[r] = -np.inf
        elif kind == "one_left":
            v = x[r, V // 3]
            x[r] = -np.inf
            x[r, V // 3] = v
        elif kind == "lowest":
            x[r, ::2] = low
        elif kind == "half_masked":
            x[r, : V // 2] = -np.inf
        elif kind == "nan":
            x[r, V // 2] = np.nan
        elif kind == "inf":
            x[r, V - 1] = np.inf
        elif kind == "few_values":
            x[r] = rng.integers(0, 3, V)
        elif kind == "peak":
            x[r, V // 2] = 60.0
        elif kind == "few_left":                            # fewer than the alternatives asked for
            keep = np.array([0, V // 2, V - 1])
            v = x[r, keep]
            x[r] = -np.inf
            x[r, keep] = v
        elif kind == "crowded":                             # the largest values all with a few threads
            x[r] *= 0.1
            i = np.arange(V)
            x[r] = np.where(i // 8 % 128 < 3, 5.0 + 4.0 * i / V, x[r])
        elif kind == "ties":                                # three larger values, then hundreds of equal ones
            x[r] = np.minimum(x[r], 2.0)
            x[r, [V // 5, V // 4, V - 1]] = [7.0, 9.0, 8.0]
        elif kind == "signed_zeros":
            x[r] = np.where(rng.random(V) < 0.5, 0.0, -0.0)
    return torch.from_numpy(x).to(dtype)


def _place(x, pad, shift):
    """x in rows of V + pad elements that start `shift` elements after an aligned address."""
    rows, V = x.shape
    hold = torch.full((rows * (V + pad) + shift + 64,), 7.0, dtype=x.dtype, device="cuda")
    view = hold[shift:shift + rows * (V + pad)].view(rows, V + pad)
    view[:, :V].copy_(x)
    return hold, view


def _in_fp32_range(v):
    """A value past fp32's largest rounds to an infinity (the type's lowest value over a temperature below 1)."""
    with np.errstate(all="ignore"):
        return np.where(np.abs(v) > float(np.finfo(np.float32).max), np.sign(v) * np.inf, v)


def _oracle(x, tau, targets, k):
    """lse, log p of targets, entropy, top ids and log p in 64 bits."""
    x = x.float().numpy().astype(np.float64)
    with np.errstate(all="ignore"):
        z = _in_fp32_range(x / tau)
        m = z.max(1)
        empty, bad = m == -np.inf, ~(m < np.inf)
        m0 = np.where(empty | bad, 0.0, m)
        d = z - m0[:, None]
        e = np.exp(d)
        log_s = np.log(e.sum(1))
        logp = d - log_s[:, None]
        p = e / e.sum(1)[:, None]
        H = -np.where(p > 0, p * logp, 0.0).sum(1)

    def settle(v, nothing):
        v = np.where(empty.reshape(-1, *([1] * (v.ndim - 1))), nothing, v)
        return np.where(bad.reshape(-1, *([1] * (v.ndim - 1))), np.nan, v)

    logp, H, lse = settle(logp, -np.inf), settle(H, 0.0), settle(m0 + log_s, -np.inf)
    rank = np.where(np.isnan(x), np.inf, x)
    nan_first = np.where(np.isnan(x), 0, 1)
    ids = np.stack([np.lexsort((np.arange(x.shape[1]), -(rank[r] + 0.0), nan_first[r]))[:k] for r in range(len(x))])
    t = np.maximum(targets, 0)
    tp = np.where(targets < 0, 0.0, np.take_along_axis(logp, t[:, None], 1)[:, 0])
    return dict(lse=lse, logp=tp, entropy=H, ids=ids, top=np.take_along_axis(logp, ids, 1), z=z, all=logp)


def _close(got, want, tol, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    want = _in_fp32_range(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    far = ~np.isfinite(want)
    assert np.array_equal(got[far & ~np.isnan(want)], want[far & ~np.isnan(want)]), what
    over = np.where(far, 0.0, np.abs(np.where(far, 0.0, got) - np.where(far, 0.0, want)) - tol)
    assert np.max(over) <= 0, (what, float(np.max(over)), np.unravel_index(np.argmax(over), over.shape))


def _spread(o):
    """Z of the module's bound, for each row."""
    with np.errstate(all="ignore"):
        m = o["z"].max(1)
        near = np.where(np.isfinite(o["z"]) & (o["z"] >= m[:, None] - 40), np.abs(o["z"]), 0.0)
    return np.where(np.isfinite(m), near.max(1), 0.0)


def _check_forward(x, tau, k, pad=0, shift=0, seed=0, only=("logp", "entropy", "lse")):
    from decoder_only_transformer_sm_b200 import native
    R, V = x.shape
    rng = np.random.default_rng(seed)
    targets = rng.integers(0, V, R).astype(np.int32)
    targets[rng.random(R) < 0.2] = -1
    o = _oracle(x, tau, targets, k)
    _, dx = _place(x, pad, shift)
    out = {n: torch.full((R + 1,), 9.0, device="cuda") for n in only}
    ids = torch.full((R + 1, k), 99, dtype=torch.int32, device="cuda") if k else None
    top = torch.full((R + 1, k), 9.0, device="cuda") if k else None
    status = native.token_logprobs(dx, V, tau, targets=torch.from_numpy(targets).cuda() if "logp" in only else None,
                                   **{n: v[:R] for n, v in out.items()}, top_ids=ids[:R] if k else None,
                                   top_logp=top[:R] if k else None)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    Z = _spread(o)
    Ds = 6 * EPS * Z + 2.0 ** -21 + (V / 128 + 16) * EPS
    got = {n: v[:R].cpu().numpy() for n, v in out.items()}
    fin = {n: np.where(np.isfinite(o[n]), np.abs(o[n]), 0.0) for n in ("lse", "logp", "entropy")}
    if "lse" in only:
        _close(got["lse"], o["lse"], Ds + 3 * EPS * (fin["lse"] + Z), "lse")
    if "logp" in only:
        _close(got["logp"], o["logp"], Ds + 6 * EPS * (2 * fin["logp"] + Z), "logp")
    if "entropy" in only:
        _close(got["entropy"], o["entropy"], (fin["entropy"] + 3) * Ds * 2 + 3 * EPS * fin["entropy"], "entropy")
    if k:
        np.testing.assert_array_equal(ids[:R].cpu().numpy(), o["ids"])
        tol = Ds[:, None] + 6 * EPS * (2 * np.where(np.isfinite(o["top"]), np.abs(o["top"]), 0.0) + Z[:, None])
        _close(top[:R].cpu().numpy(), o["top"], tol, "top_logp")
        assert torch.all(ids[R] == 99) and torch.all(top[R] == 9.0)
    assert all(v[R] == 9.0 for v in out.values())
    return o, dx, targets


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 31, 32, 33, 100, 255, 1021, 1024, 2048, 4097, 8191, 16384, 50257, 70001])
@pytest.mark.parametrize("k", [0, 1, 5, 9, 32])
def test_every_kind_of_row(dtype, V, k):
    x = _rows(KINDS * 2, V, dtype, V + k)
    _check_forward(x, 1.0, min(k, V), pad=-V % 8, seed=V)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R", [1, 2, 5, 9, 40, 75, 149, 300, 700, 1300])
@pytest.mark.parametrize("V", [700, 5003, 50257, 70001])
def test_row_counts(dtype, R, V):
    """Few rows are split over more blocks than many; many short ones take a warp each."""
    kinds = [KINDS[(i * 5) % len(KINDS)] for i in range(R)]
    if V > 6000:
        kinds = kinds[:330 if V > 60000 and R == 1300 else 150]
    _check_forward(_rows(kinds, V, dtype, R), 0.8, 5, pad=-V % 8, seed=R)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [33, 65, 200, 300, 511, 700, 1021, 2049, 4096])
@pytest.mark.parametrize("k", [9, 20, 32])
def test_many_short_rows_with_many_alternatives(dtype, V, k):
    """1203 rows: a warp takes a whole one, the last block has three."""
    kinds = [KINDS[(i * 5) % len(KINDS)] for i in range(1203)]
    _check_forward(_rows(kinds, V, dtype, V + k), 0.9, k, pad=V % 3, seed=V)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tau", [0.05, 0.7, 1.0, 3.0])
@pytest.mark.parametrize("pad,shift", [(0, 0), (1, 0), (3, 1), (8, 5), (64, 8)])
def test_temperatures_strides_and_starts(dtype, tau, pad, shift):
    for V in (333, 5003):
        _check_forward(_rows(KINDS, V, dtype, pad), tau, 7, pad=pad, shift=shift, seed=shift)


@pytest.mark.parametrize("only", [("logp",), ("entropy",), ("lse",), ()])
@pytest.mark.parametrize("V", [600, 9000])
def test_single_outputs(only, V):
    _check_forward(_rows(KINDS, V, torch.float32, 3), 1.0, 0 if only else 9, only=only)


def test_one_element_at_every_place():
    """The largest logit at each position of a row in turn: the blocks' and vectors' edges."""
    V = 1037
    x = torch.full((V, V), -2.0)
    x[torch.arange(V), torch.arange(V)] = 4.0
    for dtype in (torch.float32, torch.bfloat16):
        o, _, _ = _check_forward(x.to(dtype), 1.0, 3, pad=3, shift=1)
        assert np.array_equal(o["ids"][:, 0], np.arange(V))


@pytest.mark.parametrize("rows", [1, 297])
def test_long_rows(rows):
    """A vocabulary of millions: one row over a cluster, many a block each."""
    from decoder_only_transformer_sm_b200 import native
    V = 20_000_003 if rows == 1 else 1_000_001
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn((rows, V), generator=g, device="cuda")
    lse, H = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ids, top = torch.empty((rows, 32), dtype=torch.int32, device="cuda"), torch.empty((rows, 32), device="cuda")
    native.token_logprobs(x, V, 1.0, lse=lse, entropy=H, top_ids=ids, top_logp=top)
    for r in range(0, rows, 74):
        logp = torch.log_softmax(x[r].double(), 0)
        best = torch.sort(x[r], descending=True, stable=True).indices[:32]
        assert torch.equal(ids[r].long(), best)
        # V / 128 + 16 additions in a row at 2^-24 (V / 1024 over a cluster), exp's 2^-21
        tol = (V / (1024 if rows == 1 else 256) + 16) * EPS + 2.0 ** -21 + 40 * EPS
        assert (top[r].double() - logp[best]).abs().max() <= tol
        assert abs(float(lse[r].double() - torch.logsumexp(x[r].double(), 0))) <= tol
        want = float(-(logp.exp() * logp).sum())
        assert abs(float(H[r]) - want) <= 2 * (want + 3) * tol


def test_bad_targets_are_reported():
    from decoder_only_transformer_sm_b200 import native
    V = 50
    x = torch.randn((4, V), generator=torch.Generator().manual_seed(0)).cuda()
    t = torch.tensor([3, V, -2, -1], dtype=torch.int32, device="cuda")
    logp, lse = torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
    status = native.token_logprobs(x, V, 1.0, targets=t, logp=logp, lse=lse)
    assert int(status.item()) == 1
    want = torch.log_softmax(x.double(), 1)
    assert torch.allclose(logp[:3].double(), want[torch.arange(3), [3, V - 1, 0]], atol=1e-6) and logp[3] == 0
    status = native.token_logprobs_bwd(x, V, 1.0, lse, torch.empty_like(x), targets=t, dlogp=torch.ones(4, device="cuda"))
    assert int(status.item()) == 1


def _check_backward(x, tau, pad=0, shift=0, seed=0, use=("logp", "entropy"), in_place=False, dpad=None, dshift=None):
    from decoder_only_transformer_sm_b200 import native
    R, V = x.shape
    rng = np.random.default_rng(seed)
    targets = rng.integers(0, V, R).astype(np.int32)
    targets[rng.random(R) < 0.3] = -1
    g = rng.standard_normal(R).astype(np.float32) if "logp" in use else None
    h = (rng.standard_normal(R) * (rng.random(R) < 0.6)).astype(np.float32) if "entropy" in use else None
    o = _oracle(x, tau, targets, 1)
    lse, H = o["lse"].astype(np.float32), o["entropy"].astype(np.float32)
    hold, dx = _place(x, pad, shift)
    if in_place:
        dhold, dd = hold, dx
    else:
        pad, shift = pad if dpad is None else dpad, shift if dshift is None else dshift   # of dlogits from here on
        dhold, dd = _place(torch.full_like(x, 7.0), pad, shift)
    cu = lambda v: None if v is None else torch.from_numpy(v).cuda()  # noqa: E731
    status = native.token_logprobs_bwd(dx, V, tau, cu(lse), dd, targets=cu(targets) if g is not None else None,
                                       dlogp=cu(g), entropy=cu(H) if h is not None else None, dentropy=cu(h))
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    gg = np.where(targets >= 0, g if g is not None else 0.0, 0.0).astype(np.float64)[:, None]
    hh = (h if h is not None else np.zeros(R)).astype(np.float64)[:, None]
    L, Hd = lse.astype(np.float64)[:, None], H.astype(np.float64)[:, None]
    with np.errstate(all="ignore"):
        logp = o["z"] - L
        p = np.where(L == -np.inf, 0.0, np.exp(logp))
        inner = gg + np.where(hh != 0, hh * (np.where(p == 0, 0.0, logp) + Hd), 0.0)
        want = -np.where(p == 0, 0.0, p * inner)
        logp = np.where(L == -np.inf, 0.0, logp)
        size = np.where(np.isfinite(logp), np.abs(logp), 0.0) + np.where(np.isfinite(L), np.abs(L), 0.0)
        size = np.minimum(size, 2 * np.where(np.isfinite(L), np.abs(L), 0.0) + 110.0)
        tol = np.where(p == 0, 0.0, np.abs(want) * (6 * EPS * 2 * size + 2.0 ** -21 + 4 * EPS) + p *
                       (np.abs(hh) * 6 * EPS * (2 * size + np.abs(Hd)) + 3 * EPS * (np.abs(gg) + np.abs(hh) * (size + np.abs(Hd)))))
        tol = tol + np.where(p == 0, 0.0, 2.0 ** -126 * np.abs(inner))   # p flushed to zero
    one = np.zeros_like(want)
    one[np.arange(R), np.maximum(targets, 0)] = 1.0
    want = np.where(L == -np.inf, 0.0, want + one * gg)
    want = np.where((gg == 0) & (hh == 0), 0.0, want) / tau
    tol = np.where((gg == 0) & (hh == 0), 0.0, tol)
    tol = tol / tau + 3 * EPS * np.abs(want) + 1e-37
    if x.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * 1.01 * np.abs(want)
    _close(dd[:, :V].float().cpu().numpy(), want, tol, "dlogits")
    left = dhold.clone()
    left[shift:shift + R * (V + pad)].view(R, V + pad)[:, :V] = 7.0
    assert torch.all(left == 7.0)
    if not in_place:
        assert torch.equal(torch.nan_to_num(dx[:, :V].float().cpu(), nan=3.5), torch.nan_to_num(x.float(), nan=3.5))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 33, 255, 1021, 4097, 50257])
@pytest.mark.parametrize("use", [("logp", "entropy"), ("logp",), ("entropy",)])
def test_gradient_of_every_kind_of_row(dtype, V, use):
    _check_backward(_rows(KINDS * 2, V, dtype, V), 0.9, pad=-V % 8, seed=V, use=use)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R", [1, 3, 37, 301, 2501])
@pytest.mark.parametrize("V", [3, 65, 500, 1005, 2040, 3989])
def test_gradient_row_counts(dtype, R, V):
    """Short rows share a block, which the last of them need not fill; few rows are split."""
    kinds = [KINDS[(i * 5) % len(KINDS)] for i in range(R)]
    _check_backward(_rows(kinds, V, dtype, R), 1.1, pad=1, seed=R)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad,shift", [(0, 0), (1, 0), (3, 1), (8, 5)])
@pytest.mark.parametrize("in_place", [False, True])
def test_gradient_strides_starts_and_in_place(dtype, pad, shift, in_place):
    for R, V in ((1, 333), (40, 5003), (400, 64)):
        kinds = [KINDS[i % len(KINDS)] for i in range(R)]
        _check_backward(_rows(kinds, V, dtype, pad), 1.3, pad=pad, shift=shift, seed=shift, in_place=in_place)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad,shift,dpad,dshift", [(0, 0, 1, 0), (3, 0, 0, 1), (8, 2, 8, 3), (1, 1, 5, 0)])
def test_gradient_laid_out_apart_from_the_logits(dtype, pad, shift, dpad, dshift):
    for R, V in ((2, 50), (30, 5003)):
        kinds = [KINDS[i % len(KINDS)] for i in range(R)]
        _check_backward(_rows(kinds, V, dtype, pad), 0.8, pad=pad, shift=shift, dpad=dpad, dshift=dshift)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_far_apart(dtype):
    """Offsets past 32 bits: three rows 2^30 + 8 elements apart, forward and gradient."""
    from decoder_only_transformer_sm_b200 import native
    V, ld = 5000, (1 << 30) + 8
    hold = torch.empty(2 * ld + V, dtype=dtype, device="cuda")
    x = hold.as_strided((3, V), (ld, 1))
    x.copy_(torch.randn((3, V), generator=torch.Generator().manual_seed(1)).to(dtype))
    t = torch.tensor([1, 4999, 77], dtype=torch.int32, device="cuda")
    logp, lse = torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    ids, top = torch.empty((3, 2), dtype=torch.int32, device="cuda"), torch.empty((3, 2), device="cuda")
    native.token_logprobs(x, V, 1.0, targets=t, logp=logp, lse=lse, top_ids=ids, top_logp=top)
    near = x.clone()
    want = torch.log_softmax(near.double(), 1)
    assert torch.all((logp.double() - want.gather(1, t.long()[:, None])[:, 0]).abs() < 2e-5)
    assert torch.equal(ids.long(), torch.sort(near.float(), dim=1, descending=True, stable=True).indices[:, :2])
    g = torch.tensor([1.0, -2.0, 0.5], device="cuda")
    native.token_logprobs_bwd(x, V, 1.0, lse, x, targets=t, dlogp=g)
    grad = -g.double()[:, None] * want.exp()
    grad[torch.arange(3), t.long()] += g.double()
    assert torch.all((x.double() - grad).abs() <= 2.0 ** -8 * 1.01 * grad.abs() + 1e-6)


def test_gradient_against_differences():
    """dlogits of sum_r (a_r log p_r + b_r H_r) against central differences of the 64-bit oracle's value (step 1e-4:
    the third derivative's term is below 1e-8)."""
    from decoder_only_transformer_sm_b200 import native
    R, V, tau, step = 3, 19, 0.8, 1e-4
    rng = np.random.default_rng(5)
    x = torch.from_numpy((rng.standard_normal((R, V)) * 2).astype(np.float32))
    x[1, 4] = float("-inf")
    t = np.array([3, 7, -1], np.int32)
    a, b = rng.standard_normal(R).astype(np.float32), rng.standard_normal(R).astype(np.float32)
    dev = x.cuda()
    lse, H, logp = (torch.empty(R, device="cuda") for _ in range(3))
    native.token_logprobs(dev, V, tau, targets=torch.from_numpy(t).cuda(), logp=logp, entropy=H, lse=lse)
    d = torch.empty_like(dev)
    native.token_logprobs_bwd(dev, V, tau, lse, d, targets=torch.from_numpy(t).cuda(), dlogp=torch.from_numpy(a).cuda(),
                              entropy=H, dentropy=torch.from_numpy(b).cuda())

    def value(y):
        with np.errstate(all="ignore"):
            z = y / tau
            lp = z - np.log(np.exp(z - z.max(1, keepdims=True)).sum(1, keepdims=True)) - z.max(1, keepdims=True)
            h = -np.where(np.exp(lp) > 0, np.exp(lp) * lp, 0.0).sum(1)
        return sum(float(b[r]) * h[r] + (float(a[r]) * lp[r, t[r]] if t[r] >= 0 else 0.0) for r in range(R))

    y = x.double().numpy()
    for r in range(R):
        for v in range(V):
            if not np.isfinite(y[r, v]):
                assert d[r, v] == 0
                continue
            up, down = y.copy(), y.copy()
            up[r, v] += step
            down[r, v] -= step
            assert abs((value(up) - value(down)) / (2 * step) - float(d[r, v])) < 2e-6, (r, v)


def test_scoring_a_model_and_its_draws():
    """The operators in a row: the loss of gpt2_forward is the mean of -logp over its logits; tokens drawn by
    gpt2k_sample get the log-probability of the distribution that they were drawn from; the logits of an 8-bit lm_head
    on ln_f's output score alike."""
    from decoder_only_transformer_sm_b200 import native, synthetic as S
    s = S.ModelShape(n_layer=1, n_head=2, n_embd=128, vocab_size=1024, block_size=64)
    B, T, V = 3, 50, 1024
    idx, tgt = S.uniform_tokens(B, T, V, seed=4)
    tgt[0, :20] = -1
    for precision, dtype in (("fp32", torch.float32), ("bf16", torch.bfloat16)):
        flat = S.random_params(s, seed=5)
        m = native.GPT2(s.n_layer, s.n_head, s.n_embd, V, s.block_size, B, T, precision=precision)
        m.set_params(flat)
        logits = torch.empty((B * T, V), dtype=dtype, device="cuda")
        di, dt = torch.from_numpy(idx).cuda(), torch.from_numpy(tgt).cuda()
        torch.cuda.synchronize()
        loss = m.forward(di, dt, logits)
        logp, lse, H = (torch.empty(B * T, device="cuda") for _ in range(3))
        native.token_logprobs(logits, V, 1.0, targets=dt.reshape(-1), logp=logp, lse=lse, entropy=H)
        mean = float(-logp.double().sum() / (dt >= 0).sum())
        # fp32: the same logits, log sums within 1e-6 each; bf16: the loss path rounds the same logits to bf16
        assert abs(mean - loss) <= 2e-6 * abs(loss), (mean, loss)
        # draws at a temperature, scored at the same one
        tau = 0.8
        u = torch.rand(B * T, generator=torch.Generator().manual_seed(2)).cuda()
        drawn = torch.empty(B * T, dtype=torch.int32, device="cuda")
        native.sample(logits, V, tau, 0, u, drawn)
        native.token_logprobs(logits, V, tau, targets=drawn, logp=logp)
        want = torch.log_softmax(logits.double() / tau, 1).gather(1, drawn.long()[:, None])[:, 0]
        assert torch.all((logp.double() - want).abs() <= 2e-5)
        # the 8-bit lm_head: wte's rows by output channel, ln_f's output by token
        x = torch.from_numpy(m.debug_activation("ln_f", 0, B, T).reshape(B * T, -1)).cuda()
        m.close()
        wte = torch.from_numpy(flat[:V * s.n_embd].reshape(V, s.n_embd).astype(np.float32)).cuda()
        wq, ws = torch.empty(wte.shape, dtype=torch.int8, device="cuda"), torch.empty(V, device="cuda")
        xq, xs = torch.empty(x.shape, dtype=torch.int8, device="cuda"), torch.empty(B * T, device="cuda")
        native.quantize_rows(wte, wq, ws)
        native.quantize_rows(x, xq, xs)
        l8 = torch.empty((B * T, V), dtype=dtype, device="cuda")
        native.matmul_i8(xq, xs, wq, ws, l8)
        ids, top = torch.empty((B * T, 5), dtype=torch.int32, device="cuda"), torch.empty((B * T, 5), device="cuda")
        native.token_logprobs(l8, V, 1.0, targets=dt.reshape(-1), logp=logp, lse=lse, top_ids=ids, top_logp=top)
        exact = (xq.double() @ wq.double().t()) * xs.double()[:, None] * ws.double()
        bound = exact.abs() * (3 * EPS + (2.0 ** -8 if dtype == torch.bfloat16 else 0.0))
        assert torch.all((l8.double() - exact).abs() <= bound * 1.01)
        want = torch.log_softmax(l8.double(), 1)
        picked = want.gather(1, dt.reshape(-1).long().clamp(min=0)[:, None])[:, 0]
        assert torch.all((logp.double() - torch.where(dt.reshape(-1) < 0, 0.0, picked)).abs() <= 2e-5)
        assert torch.equal(ids.long(), torch.sort(l8.float(), dim=1, descending=True, stable=True).indices[:, :5])
        assert torch.all((top.double() - want.gather(1, ids.long())).abs() <= 2e-5)


def test_side_stream_and_graphs():
    """Forward and gradient captured into two graphs, replayed interleaved on new logits and on a side stream,
    bit-equal to direct calls."""
    from decoder_only_transformer_sm_b200 import native
    R, V = 6, 9001
    gen = torch.Generator().manual_seed(0)

    class Loss:
        def __init__(self):
            self.x = torch.zeros((R, V), dtype=torch.bfloat16, device="cuda")
            self.t = torch.arange(R, dtype=torch.int32, device="cuda") * 700
            self.logp, self.H, self.lse = (torch.empty(R, device="cuda") for _ in range(3))
            self.ids = torch.empty((R, 4), dtype=torch.int32, device="cuda")
            self.top = torch.empty((R, 4), device="cuda")
            self.g = torch.full((R,), -1.0 / R, device="cuda")
            self.d = torch.empty_like(self.x)
            self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

        def run(self, stream=None):
            native.token_logprobs(self.x, V, 1.0, targets=self.t, logp=self.logp, entropy=self.H, lse=self.lse,
                                  top_ids=self.ids, top_logp=self.top, status=self.status, stream=stream)
            native.token_logprobs_bwd(self.x, V, 1.0, self.lse, self.d, targets=self.t, dlogp=self.g, entropy=self.H,
                                      dentropy=self.g, status=self.status, stream=stream)

        def results(self):
            return [v.clone() for v in (self.logp, self.H, self.lse, self.ids, self.top, self.d)]

    xs = [torch.randn((R, V), generator=gen).to(torch.bfloat16).cuda() for _ in range(4)]
    want = []
    for x in xs:
        loss = Loss()
        loss.x.copy_(x)
        loss.run()
        want.append(loss.results())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    loss = Loss()
    loss.x.copy_(xs[1])
    side.wait_stream(torch.cuda.current_stream())
    loss.run(stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(loss.results(), want[1]))
    made = []
    for _ in range(2):
        loss, graph = Loss(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            loss.run()
        made.append((loss, graph))
    for i in (0, 2):
        for j, (loss, graph) in enumerate(made):
            loss.x.copy_(xs[i + j])
            graph.replay()
        for j, (loss, _) in enumerate(made):
            assert all(torch.equal(a, b) for a, b in zip(loss.results(), want[i + j]))


def test_calls_at_once_on_two_streams():
    """An 8-bit product, quantisation and log-probabilities on one stream beside the same on another: each gets what
    it gets alone."""
    from decoder_only_transformer_sm_b200 import native
    gen = torch.Generator().manual_seed(3)

    class Work:
        def __init__(self, M, N, K, V):
            self.x = torch.randn((M, K), generator=gen).to(torch.bfloat16).cuda()
            self.q, self.s = torch.empty((M, K), dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
            self.w = torch.randint(-127, 128, (N, K), generator=gen, dtype=torch.int8).cuda()
            self.ws = torch.rand(N, generator=gen).cuda() * 1e-3
            self.out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
            self.V = V
            self.H, self.lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
            self.ids, self.top = torch.empty((M, 9), dtype=torch.int32, device="cuda"), torch.empty((M, 9), device="cuda")
            self.d = torch.empty_like(self.out)
            self.g = torch.rand(M, generator=gen).cuda()
            self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

        def run(self, stream=None):
            native.quantize_rows(self.x, self.q, self.s, stream=stream)
            native.matmul_i8(self.q, self.s, self.w, self.ws, self.out, status=self.status, stream=stream)
            native.token_logprobs(self.out, self.V, 0.9, lse=self.lse, entropy=self.H, top_ids=self.ids,
                                  top_logp=self.top, status=self.status, stream=stream)
            native.token_logprobs_bwd(self.out, self.V, 0.9, self.lse, self.d, entropy=self.H, dentropy=self.g,
                                      status=self.status, stream=stream)

        def results(self):
            return [v.clone() for v in (self.q, self.s, self.out, self.H, self.lse, self.ids, self.top, self.d[:, :self.V])]

    works = [Work(1500, 9000, 512, 8999), Work(40, 30000, 768, 29990), Work(5, 50304, 768, 50257), Work(300, 1000, 99, 1000)]
    want = []
    for w in works:
        w.run()
        want.append(w.results())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in works]
    for _ in range(10):
        for w, s in zip(works, streams):
            w.run(stream=s.cuda_stream)
    torch.cuda.synchronize()
    for w, r in zip(works, want):
        assert int(w.status.item()) == 0
        assert all(torch.equal(a, b) for a, b in zip(w.results(), r))


@pytest.mark.parametrize("dtype,V", [(torch.float32, 32768), (torch.float32, 50257), (torch.bfloat16, 65536),
                                     (torch.bfloat16, 70001)])
@pytest.mark.parametrize("k", [9, 24, 25, 32])
def test_largest_values_of_many_long_rows_with_few_threads(dtype, V, k):
    """Rows of 120 KB and more, a block of 256 threads each (more rows than SMs): each warp's list of alternatives has
    room, where the allowed, or just the largest, values lie side by side or all with a few of the threads."""
    from decoder_only_transformer_sm_b200 import native
    N = 16 // torch.tensor([], dtype=dtype).element_size()      # of a vector; vectors go to the 256 threads in turn
    rng = np.random.default_rng(V + k)
    i = np.arange(V)
    chosen = [(i >= 1000) & (i < 1240), (i >= V - 700) & (i < V - 400)]
    chosen += [i // N % 256 < n for n in (1, 8, k - 1, k, 40)] + [(i // N % 256 % 8 == 3) & (i // N % 256 < 8 * (k - 1))]
    kinds = []
    for c in chosen:
        noise = rng.standard_normal(V)
        kinds += [np.where(c, noise, -np.inf), np.where(c, 6.0 + noise, 0.1 * noise)]
    x = torch.from_numpy(np.stack(kinds).astype(np.float32)).to(dtype)
    R = len(kinds) * 11                                         # 176 rows: not split
    o = _oracle(x, 1.0, np.zeros(len(kinds), np.int64), k)
    ids, top = torch.empty((R, k), dtype=torch.int32, device="cuda"), torch.empty((R, k), device="cuda")
    lse = torch.empty(R, device="cuda")
    _, dx = _place(x.repeat(11, 1), -V % 8, 0)
    native.token_logprobs(dx, V, 1.0, lse=lse, top_ids=ids, top_logp=top)
    np.testing.assert_array_equal(ids.cpu().numpy(), np.tile(o["ids"], (11, 1)))
    # 256 threads: V / 512 additions of a pair's sum, 5 + 8 joins
    Z = np.tile(_spread(o), 11)
    tol = 6 * EPS * Z + 2.0 ** -21 + (V / 512 + 16) * EPS
    _close(lse.cpu().numpy(), np.tile(o["lse"], 11), tol + 3 * EPS * (np.abs(np.tile(o["lse"], 11)) + Z), "lse")
    want = np.tile(o["top"], (11, 1))
    size = np.where(np.isfinite(want), np.abs(want), 0.0)
    _close(top.cpu().numpy(), want, tol[:, None] + 6 * EPS * (2 * size + Z[:, None]), "top_logp")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,V", [(5, 40), (5, 3000), (5, 50257), (160, 5003), (160, 70001)])
def test_rows_whose_scaled_logits_all_overflow(dtype, R, V):
    """Finite logits below -1.8e38 at temperature 0.5: every z is -inf, so nothing is left of the row; the alternatives
    are still the largest logits, -inf after them."""
    rng = np.random.default_rng(V)
    x = rng.uniform(-3.3e38, -1.8e38, (5, V)).astype(np.float32)
    x[1] = -2e38
    x[2, ::2] = -np.inf
    x[3, 2:] = -np.inf
    x[4] = np.finfo(np.float32).min if dtype == torch.float32 else -3e38
    o, _, _ = _check_forward(torch.from_numpy(np.tile(x, (R // 5, 1))).to(dtype), 0.5, 9, pad=-V % 8, seed=R)
    assert np.all(o["lse"] == -np.inf) and list(o["ids"][3][:2]) in ([0, 1], [1, 0])
    _check_backward(torch.from_numpy(x).to(dtype), 0.5, pad=-V % 8)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tau", [1e-30, 1e-4, 1e6, 1e20])
@pytest.mark.parametrize("R,V", [(16, 300), (16, 9000), (160, 5003), (160, 70001)])
def test_temperatures_of_every_size(dtype, tau, R, V):
    """Logits of the temperature's size, with the type's lowest values and (last row) differences that fp32 does not
    hold among them."""
    kinds = KINDS * (R // len(KINDS)) if V < 60000 else KINDS[:8] * (R // 8)
    x = _rows(kinds, V, torch.float32, R)
    low = torch.tensor(torch.finfo(dtype).min, dtype=torch.float32)
    x = torch.where(x <= -3e38, torch.where(x.isinf(), x, low), x * tau)
    if V == 300:
        _check_backward(x.to(dtype), tau, pad=-V % 8, seed=V)
    x[-1, 0], x[-1, 1], x[-1, 2] = -1e32, -low, low
    if tau < 1:
        x[-1, 1] = 1e32 * tau                               # (the largest over tau would be infinite)
    _check_forward(x.to(dtype), tau, 6, pad=-V % 8, seed=V)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,V", [(3, 40), (3, 40000), (160, 5003), (160, 70001)])
def test_a_token_further_below_the_largest_than_fp32_reaches(dtype, R, V):
    """A forbidden token at the type's lowest value beside a largest one near its largest: their difference is no fp32
    number, divided by the temperature it is."""
    from decoder_only_transformer_sm_b200 import native
    high, low = float(torch.finfo(dtype).max), float(torch.finfo(dtype).min)
    x = torch.full((R, V), low, dtype=dtype)
    x[:, 7] = high
    x[:, 20:] = float("-inf")
    t = torch.full((R,), 3, dtype=torch.int32, device="cuda")
    for tau in (1.0, 3.0, 1e6, 1e20):
        logp, H, lse = (torch.empty(R, device="cuda") for _ in range(3))
        ids, top = torch.empty((R, 22), dtype=torch.int32, device="cuda"), torch.empty((R, 22), device="cuda")
        native.token_logprobs(x.cuda(), V, tau, targets=t, logp=logp, entropy=H, lse=lse, top_ids=ids, top_logp=top)
        gap = _in_fp32_range(np.float64((low - high) / tau))
        want = np.full((R, 22), -np.inf)
        want[:, 0], want[:, 1:20] = 0.0, gap
        size = np.where(np.isfinite(want), np.abs(want), 0.0)
        _close(top.cpu().numpy(), want, 6 * EPS * size, "top_logp")
        _close(logp.cpu().numpy(), np.full(R, gap), 6 * EPS * size[0, 1], "logp")
        _close(lse.cpu().numpy(), np.full(R, high / tau), 6 * EPS * high / tau, "lse")
        assert torch.all(H == 0) and ids[0].tolist() == [7] + [v for v in range(20) if v != 7] + [20, 21]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tau", [1.0, 0.7])
@pytest.mark.parametrize("R,V", [(12, 3), (12, 40), (12, 2000), (1200, 5003), (48, 5003), (12, 50257), (156, 16384), (156, 70001)])
def test_log_probability_of_a_sure_token(dtype, tau, R, V):
    """A token that has nearly all of the probability: with r the sum of all others over it, its log-probability is
    -log(1 + r), near -r, and right relative to that, however small r is; and so is the entropy, log(1 + r) + sum of the
    others' (m - z) / (1 + r), two numbers of one sign. Relative errors, eps = 2^-24: a term of r has 4 eps of its exponent
    (d = x - m, 1 / tau, log2(e) / tau, their product), exp's 2^-21; the additions, all of one sign, an eps each (a warp
    sums V / 64 in a row, 128 and 256 threads fewer), the joins 16; the logarithm and the last operations 6."""
    from decoder_only_transformer_sm_b200 import native
    rng = np.random.default_rng(V + R)
    x = rng.standard_normal((12, V)).astype(np.float32)
    want_r = np.array([0.3, 0.07, 0.0626, 0.0624, 0.05, 4e-3, 1e-3, 1e-4, 1e-5, 1e-6, 1e-8, 1e-12])
    at = rng.integers(0, V, 12)
    at[:3] = 0, V - 1, V // 2
    others = np.arange(V)[None, :] != at[:, None]
    x[::3] = np.where(others[::3] & (np.arange(V) % 2 == 1), -np.inf, x[::3])       # masked tokens among the others
    x = torch.from_numpy(x).to(dtype).float().numpy().astype(np.float64)
    z0 = np.where(others, x / tau, -np.inf)
    mass = np.log(np.exp(z0).sum(1)) if V > 3 else np.log(np.maximum(np.exp(z0).sum(1), 1e-3))
    x[np.arange(12), at] = tau * (mass - np.log(want_r))
    t = torch.from_numpy(x.astype(np.float32)).to(dtype)
    x = t.double().numpy()
    m = x[np.arange(12), at][:, None]
    d = np.where(others, (x - m) / tau, -np.inf)
    e = np.exp(d)
    r = e.sum(1)
    logp, H = -np.log1p(r), np.log1p(r) - np.where(e > 0, e * np.where(e > 0, d, 0.0), 0.0).sum(1) / (1 + r)
    far = np.where(e > e.max(1, keepdims=True) * 1e-12, np.abs(np.where(e > 0, d, 0.0)), 0.0).max(1)
    adds = V / 64 if V <= 2048 or (V <= 8192 and R > 1184) else V / 256
    rel = 4 * EPS * far + 2.0 ** -21 + (adds + 16 + 6) * EPS
    rel = np.where(r > 0.0625, rel + (adds + 22) * EPS * 1.1 / np.log1p(r), rel)    # s itself is summed there
    n = R // 12
    lp, ent, lse = (torch.empty(R, device="cuda") for _ in range(3))
    ids, top = torch.empty((R, 2), dtype=torch.int32, device="cuda"), torch.empty((R, 2), device="cuda")
    targets = torch.from_numpy(np.tile(at, n).astype(np.int32)).cuda()
    _, dx = _place(t.repeat(n, 1), -V % 8, 0)
    native.token_logprobs(dx, V, tau, targets=targets, logp=lp, entropy=ent, lse=lse, top_ids=ids, top_logp=top)
    assert np.array_equal(ids[:, 0].cpu().numpy(), np.tile(at, n))
    assert torch.equal(top[:, 0], lp)
    _close(lp.cpu().numpy(), np.tile(logp, n), np.tile(rel * np.abs(logp), n), "logp")
    _close(ent.cpu().numpy(), np.tile(H, n), np.tile(rel * H + 6 * EPS * H, n), "entropy")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tau", [1.0, 0.7])
@pytest.mark.parametrize("R,V", [(12, 3), (12, 40), (300, 1000), (12, 5003), (240, 2123), (12, 50257)])
@pytest.mark.parametrize("in_place", [False, True])
def test_gradient_of_a_sure_target(dtype, tau, R, V, in_place):
    """1 - p of a target with nearly all of the probability, relative to itself: g (1 - p) = -g expm1(d) with
    d = (x - tau lse) / tau, where the subtraction rounds once (fma): 3 eps of d, expm1's 2^-22, products 3 eps; the
    entropy's part h p (d + H) as in the other gradient tests, its p 2^-21 and 4 eps of d off."""
    from decoder_only_transformer_sm_b200 import native
    rng = np.random.default_rng(V + R)
    want_r = np.array([0.3, 0.07, 0.05, 0.02, 4e-3, 1e-3, 1e-4, 3e-5])
    at = rng.integers(0, V, R)
    at[:3] = 0, V - 1, V // 2
    x = rng.standard_normal((R, V))
    others = np.arange(V)[None, :] != at[:, None]
    mass = np.log(np.where(others, np.exp(x / tau), 0.0).sum(1))
    x[np.arange(R), at] = tau * (mass - np.log(want_r[np.arange(R) % 8]))
    t = torch.from_numpy(x.astype(np.float32)).to(dtype)
    x = t.double().numpy()
    z = x / tau
    lse = np.log(np.exp(z - z.max(1, keepdims=True)).sum(1)) + z.max(1)
    p = np.exp(z - lse[:, None])
    H = (-np.where(p > 0, p * (z - lse[:, None]), 0.0).sum(1)).astype(np.float32)
    lse = lse.astype(np.float32)
    g = (rng.standard_normal(R) + 2.0).astype(np.float32)
    h = (rng.standard_normal(R) * (np.arange(R) % 3 == 0)).astype(np.float32)
    _, dx = _place(t, -V % 8, 0)
    out = dx if in_place else torch.empty_like(dx)
    cu = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    native.token_logprobs_bwd(dx, V, tau, cu(lse), out, targets=cu(at.astype(np.int32)), dlogp=cu(g), entropy=cu(H),
                              dentropy=cu(h))
    got = out[:, :V].double().cpu().numpy()[np.arange(R), at]
    tau32 = float(np.float32(tau))
    d = (x[np.arange(R), at] - tau32 * lse.astype(np.float64)) / tau32
    G, Hd, hd = g.astype(np.float64), H.astype(np.float64), h.astype(np.float64)
    want = (-G * np.expm1(d) - hd * np.exp(d) * (d + Hd)) / tau32
    tol = np.abs(G * np.expm1(d)) * (6 * EPS + 2.0 ** -22)
    tol = tol + np.abs(hd) * ((2.0 ** -21 + 4 * EPS * np.abs(d)) * np.abs(d + Hd) + 6 * EPS * (np.abs(d) + np.abs(Hd)))
    tol = tol / tau32 + (2.0 ** -8 * 1.01 if dtype == torch.bfloat16 else 2 * EPS) * np.abs(want)
    _close(got, want, tol, "dlogits of the target")


def test_stream_given_as_a_handle_or_as_a_torch_stream():
    """With and without a status tensor, as the other bindings of the library take it."""
    from decoder_only_transformer_sm_b200 import native
    x = torch.randn((3, 500), generator=torch.Generator().manual_seed(0)).cuda()
    want = torch.empty(3, device="cuda")
    native.token_logprobs(x, 500, 1.0, lse=want)
    q, s = torch.empty((3, 500), dtype=torch.int8, device="cuda"), torch.empty(3, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream, torch.cuda.default_stream(), 0):
        for status in (None, torch.zeros(1, dtype=torch.int32, device="cuda")):
            torch.cuda.synchronize()
            lse, d, out = torch.empty(3, device="cuda"), torch.empty_like(x), torch.empty((3, 3), device="cuda")
            native.quantize_rows(x, q, s, stream=stream)
            got = [native.token_logprobs(x, 500, 1.0, lse=lse, status=status, stream=stream),
                   native.token_logprobs_bwd(x, 500, 1.0, lse, d, entropy=lse, dentropy=lse, status=status, stream=stream),
                   native.matmul_i8(q, s, q, s, out, status=status, stream=stream)]
            torch.cuda.synchronize()
            assert torch.equal(lse, want) and all(int(v.item()) == 0 for v in got)
