"""GPU parity of the drafter-training operators against their definitions in 64 bits
(train_oracle.py, which derives the tolerances), at the sizes and masks where they can go wrong."""
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import lossless_draft_verification_row_amd as L
from lossless_draft_verification_row_amd import workloads as W
import harness as H
import train_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def note(msg):
    print(msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module", autouse=True)
def _gpu_ready():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm GPU")
    L.load_library()


def n64(t):
    return t.detach().double().cpu().numpy()


def rows_of(R, V, dt, seed, sigma=3.0):
    """Rows of N(0, sigma^2) with a few favoured tokens, in a type."""
    rng = np.random.default_rng(seed)
    x = rng.normal(0.0, sigma, (R, V))
    for r in range(R):
        hot = rng.integers(0, V, 4)
        x[r, hot] += rng.uniform(0, 10, 4)
    return torch.from_numpy(x).to(dt)


def within(got, ref, tol, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    tol = np.broadcast_to(tol, ref.shape)
    assert (np.isnan(got) == np.isnan(ref)).all(), f"{what}: NaN in other places"
    inf = np.isinf(ref)
    assert (got[inf] == ref[inf]).all(), f"{what}: infinities"
    fine = np.isfinite(ref)
    off = np.where(fine, np.abs(np.where(fine, got, 0) - np.where(fine, ref, 0)) - tol, -1.0)
    i = np.unravel_index(int(np.argmax(off)), off.shape) if off.size else None
    assert i is None or off[i] <= 0, f"{what}{i}: {got[i]} against {ref[i]}, may be {tol[i]} off"


# ---------------------------------------------------------------- spec_row_topk

def check_topk(l, K, T, **kw):
    res = L.spec_row_topk(l, K, temperature=T, **kw)
    torch.cuda.synchronize()
    index, logit, log_z = O.topk(n64(l), K, T)
    np.testing.assert_array_equal(res["index"].cpu().numpy(), index)
    np.testing.assert_array_equal(n64(res["logit"]), logit)
    within(n64(res["log_z"]), log_z, O.log_z_tolerance(log_z), "log_z")
    return res


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("R,V,K", [(1, 1, 1), (2, 5, 8), (3, 255, 256), (5, 4097, 17), (2, 8192, 128), (3, 8193, 129),
                                   (2, 16391, 256), (1, 70001, 64)])
def test_topk_sizes(R, V, K, dt):
    note(f"case topk R={R} V={V} K={K} {dt}")
    check_topk(rows_of(R, V, dt, R + V + K).to(DEV), K, 0.7)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("K", [1, 50, 256])
def test_topk_orders_and_ties(K, dt):
    """Rows whose largest logits share a thread, equal rows, rows of few values, ascending and
    descending ones, signed zeros: the lists are exact, ties by index."""
    V = 3 * 8192 + 100
    rng = np.random.default_rng(K)
    x = np.zeros((9, V))
    x[1] = np.arange(V)[::-1] / 64.0
    x[2] = np.arange(V) / 64.0
    x[3] = rng.integers(0, 3, V)
    x[4] = rng.normal(0, 1, V)
    x[4, 8192:8192 + 2048] = 50.0 + rng.integers(0, 2, 2048)     # one segment's ties
    x[5] = -rng.integers(0, 2, V) * 0.0                           # -0 and 0 are equal
    x[6] = -1e30
    x[6, rng.integers(0, V, 300)] = 1e30
    x[7] = rng.normal(0, 1, V)
    x[7, 16:24] = 9.0                                             # one thread's eight logits
    x[8, ::2] = -0.0
    check_topk(torch.from_numpy(x).to(dt).to(DEV), K, 1.0)


@pytest.mark.parametrize("dt", [BF, F32])
def test_topk_masks_and_nonfinite_rows(dt):
    V, K = 20000, 64
    l = rows_of(8, V, dt, 3)
    l[0] = -np.inf                       # nothing left
    l[1] = -np.inf
    l[1, 12345] = -3.0                   # a single token left
    l[2, :8192] = -np.inf                # a masked segment
    l[3] = -np.inf
    l[3, 100:140] = 1.5                  # fewer than K left
    l[4, 7] = np.nan
    l[5, 19999] = np.inf
    l[6] = torch.finfo(dt).min           # the type's lowest value is a logit like another
    l[6, 5] = 0.0
    l[7, 100:] = torch.finfo(dt).min
    check_topk(l.to(DEV), K, 1.0)


def test_topk_strides_and_caller_tensors():
    V, K = 9001, 40
    for dt, off in ((BF, 3), (F32, 1), (BF, 8), (F32, 4)):
        wide = torch.full((6, V + 2 * off + 16), float("nan"), dtype=dt)
        wide[:, off:off + V] = rows_of(6, V, dt, 9)
        wide = wide.to(DEV)
        out = {"index": torch.full((6, K), 7, dtype=torch.int32, device=DEV), "logit": torch.zeros((6, K), device=DEV)}
        n = L.spec_row_topk_workspace_bytes(6, V, K)
        ws = torch.full((n,), 0xA5, dtype=torch.uint8, device=DEV)     # no zero-fill is asked for
        res = check_topk(wide[:, off:off + V], K, 2.0, out=out, workspace=ws)
        assert res is out


def test_topk_of_no_rows():
    res = L.spec_row_topk(torch.empty((0, 100), device=DEV), 5)
    assert res["index"].shape == (0, 5) and res["log_z"].shape == (0,)


# ---------------------------------------------------------------- spec_topk_distill

def check_distill(s, index, t, lz, T, w, *, in_place=False, **kw):
    dev = [None if v is None else v.to(DEV) for v in (index, t, lz, w)]
    ref = O.distill(n64(s), index.numpy(), t.numpy(), None if lz is None else n64(lz), T, None if w is None else n64(w))
    only = L.spec_topk_distill(s, dev[0], dev[1], teacher_log_z=dev[2], temperature=T, row_weight=dev[3])
    assert "d_logits" not in only
    out = {"d_logits": s} if in_place else kw.pop("out", None)
    res = L.spec_topk_distill(s, dev[0], dev[1], teacher_log_z=dev[2], temperature=T, row_weight=dev[3], grad=True, out=out, **kw)
    torch.cuda.synchronize()
    loss, log_z, d, e_loss, e_d = ref
    for o in (only, res):
        within(n64(o["loss"]), loss, e_loss, "loss")
        within(n64(o["log_z"]), log_z, O.log_z_tolerance(log_z), "log_z")
    half = O.HALF[s.dtype]
    within(n64(res["d_logits"]), d, e_d + half * (np.abs(d) + e_d), "d_logits")
    return res


def teacher_of(s, K, T, seed, tail):
    """A teacher near the student: its K largest logits and, if asked, its log Z."""
    rng = np.random.default_rng(seed)
    x = n64(s) + rng.normal(0, 1, tuple(s.shape))
    x = np.where(np.isnan(x) | np.isinf(x), 0.0, x)
    k = min(K, x.shape[1])
    idx = np.argsort(-x, axis=1, kind="stable")[:, :k]
    val = np.take_along_axis(x, idx, 1)
    index, t = np.full((len(x), K), -1, np.int32), np.zeros((len(x), K), np.float32)
    index[:, :k], t[:, :k] = idx, val
    lz = None
    if tail:
        m = x.max(axis=1, keepdims=True)
        lz = torch.from_numpy((m / T + np.log(np.exp((x - m) / T).sum(axis=1, keepdims=True)))[:, 0].astype(np.float32))
    return torch.from_numpy(index), torch.from_numpy(t), lz


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("R,V,K,T", [(1, 1, 1, 1.0), (2, 7, 3, 1.0), (3, 255, 256, 0.5), (5, 4097, 17, 2.0), (2, 8192, 64, 1.0),
                                     (3, 8193, 1, 0.7), (2, 33001, 256, 1.0)])
def test_distill_sizes(R, V, K, T, tail, dt):
    note(f"case distill R={R} V={V} K={K} T={T} tail={tail} {dt}")
    s = rows_of(R, V, dt, R + V + K)
    index, t, lz = teacher_of(s, K, T, V, tail)
    w = torch.from_numpy(np.random.default_rng(1).uniform(-1, 2, R).astype(np.float32))
    check_distill(s.to(DEV), index, t, lz, T, w)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("times", [1, 33])
def test_distill_lists_and_masks(tail, dt, times):
    """(33 times over: enough rows that each workgroup takes whole ones.)  Empty, partly padded and doubled lists, tokens out of range, logits of -inf in them; student
    rows that are masked in part, in the list, off the list or wholly; NaN and +inf rows, in rows
    that count and in rows that do not."""
    R, V, K = 16, 10000, 12
    s = rows_of(R, V, dt, 77)
    index, t, lz = teacher_of(s, K, 1.0, 5, tail)
    index[0] = -1                                    # empty
    index[1, 3:] = -1                                # short
    index[2, 4] = V                                  # out of range
    index[2, 5] = 2 ** 31 - 1
    index[3, 1] = index[3, 0]                        # the same token twice
    index[3, 7] = index[3, 0]
    t[4, 2:] = -np.inf                               # no mass there
    t[5] = -np.inf                                   # none at all
    s[6, 5000:] = -np.inf                            # a masked student
    s[7, index[7].long()] = -np.inf                  # masked on the list: the loss is +inf
    keep = torch.zeros(V, dtype=torch.bool)
    keep[index[8].long()] = True
    s[8, ~keep] = -np.inf                            # masked off the list
    s[9] = -np.inf                                   # nothing left
    s[10, 17] = np.nan
    s[11, 9999] = np.inf
    s[12] = np.nan                                   # padding: garbage, empty list
    index[12] = -1
    s[13, 3] = np.nan                                # padding: garbage, weight 0
    s[14] = torch.finfo(dt).min                      # the lowest values in masked places
    s[14, index[14].long()] = 1.0
    w = torch.ones(R)
    w[13] = 0.0
    w[15] = 0.0
    lz = None if lz is None else lz.repeat(times)
    check_distill(s.repeat(times, 1).to(DEV), index.repeat(times, 1), t.repeat(times, 1), lz, 1.0, w.repeat(times))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("R,V,K", [(512, 5, 3), (515, 8, 8), (600, 4099, 40), (1100, 16389, 256)])
def test_distill_whole_rows(R, V, K, dt):
    """Enough rows that each workgroup takes whole ones: vocabularies of less than a vector, of one and
    of an odd number, rows off the 16-byte grid, in place and not."""
    note(f"case distill whole rows R={R} V={V} K={K} {dt}")
    base = rows_of(37, V, dt, V)
    index, t, lz = teacher_of(base, K, 1.0, V, True)
    rep = torch.arange(R) % 37
    w = torch.from_numpy(np.random.default_rng(1).uniform(-1, 2, R).astype(np.float32))
    wide = torch.full((R, V + 3), float("nan"), dtype=dt, device=DEV)
    for in_place in (False, True):
        wide[:, 1:1 + V] = base[rep].to(DEV)
        check_distill(wide[:, 1:1 + V], index[rep].contiguous(), t[rep].contiguous(), lz[rep].contiguous(), 1.0, w, in_place=in_place)
    assert torch.isnan(wide[:, 0]).all() and torch.isnan(wide[:, 1 + V:]).all()


def test_distill_far_apart():
    """A student whose mass off the list is below fp32's range against its largest logit, and one
    whose listed logits are: losses and gradients keep their size."""
    V, K = 9000, 4
    s = torch.zeros((2, V), dtype=F32)
    s[0] = -200.0 + torch.from_numpy(np.random.default_rng(0).normal(0, 1, V)).float()
    s[0, :4] = torch.tensor([1.0, 2.0, 0.5, 0.0])
    s[1, :4] = -150.0
    index = torch.arange(4, dtype=torch.int32).repeat(2, 1)
    t = torch.tensor([[1.0, 2.0, 0.5, 0.0]] * 2)
    lz = torch.logsumexp(t.double(), dim=1).float() + 0.3
    check_distill(s.to(DEV), index, t, lz, 1.0, None)


def test_distill_in_place_and_strides():
    V, K = 17003, 9
    for dt, off in ((BF, 1), (F32, 3), (BF, 8), (F32, 4)):
        wide = torch.full((5, V + 2 * off + 16), float("nan"), dtype=dt)
        wide[:, off:off + V] = rows_of(5, V, dt, 4)
        index, t, lz = teacher_of(wide[:, off:off + V], K, 1.0, 6, True)
        before = wide.clone()
        wide = wide.to(DEV)
        check_distill(wide[:, off:off + V], index, t, lz, 1.0, None, in_place=True)
        after = wide.cpu()
        before[:, off:off + V] = after[:, off:off + V]
        assert torch.equal(after.view(torch.int16 if dt == BF else torch.int32), before.view(torch.int16 if dt == BF else torch.int32)), \
            "wrote outside the rows"
        # gradients with another stride than the logits
        s = rows_of(5, V, dt, 8).to(DEV)
        index, t, lz = teacher_of(s, K, 1.0, 9, True)
        d = torch.empty((5, V + 24), dtype=dt, device=DEV)
        check_distill(s, index, t, lz, 1.0, None, out={"d_logits": d[:, 8:8 + V]})


def test_distill_formula_against_differences():
    """The definition's gradient against central differences of its loss, in 64 bits, and the
    kernel's against differences of its own fp32 losses along random directions."""
    rng = np.random.default_rng(11)
    V, K, T = 40, 6, 0.8
    s = rng.normal(0, 2, (3, V))
    index = np.stack([rng.permutation(V)[:K] for _ in range(3)]).astype(np.int32)
    t = rng.normal(0, 2, (3, K)).astype(np.float32)
    w = np.array([1.0, 0.5, -2.0])
    for lz in (None, np.log(np.exp(t.astype(np.float64) / T).sum(axis=1)) + 0.4):
        d = O.distill(s, index, t, lz, T, w)[2]
        for r, v in ((0, 0), (1, int(index[1, 2])), (2, int(index[2, 0])), (0, int(index[0, 5])), (2, 39)):
            e = np.zeros_like(s)
            e[r, v] = 1e-5
            diff = (w * (O.distill(s + e, index, t, lz, T, w)[0] - O.distill(s - e, index, t, lz, T, w)[0])).sum() / 2e-5
            assert abs(diff - d[r, v]) <= 1e-8      # 1e-10 (third derivative) and 2^-52 / 1e-5 of the loss
        sg, ig, tg = torch.from_numpy(s).float().to(DEV), torch.from_numpy(index).to(DEV), torch.from_numpy(t).to(DEV)
        zg = None if lz is None else torch.from_numpy(lz).float().to(DEV)
        wg = torch.from_numpy(w).float().to(DEV)
        call = lambda x: L.spec_topk_distill(x, ig, tg, teacher_log_z=zg, temperature=T, row_weight=wg, grad=True)  # noqa: E731
        base = call(sg)
        u = torch.from_numpy(rng.choice([-1.0, 1.0], s.shape)).float().to(DEV)
        h = 2.0 ** -6
        up, dn = call(sg + h * u), call(sg - h * u)
        diff = float(((up["loss"].double() - dn["loss"].double()) * wg.double()).sum()) / (2 * h)
        along = float((base["d_logits"].double() * u.double()).sum())
        # losses are off by 3 LZ each; the third derivative of a log-sum-exp along +-1 / T steps is
        # at most 8 / T^3 a row and outcome (two of them with a mass off the list)
        tol = 6 * O.LZ * 3.5 * 2 / (2 * h) + 3.5 * 2 * 8 / T ** 3 * h * h / 6
        assert abs(diff - along) <= tol


# ---------------------------------------------------------------- spec_lm_head_loss

def check_head(h, wt, y, T, w, *, strided=False, **kw):
    """h, wt bf16 on the GPU; garbage in rows that are left out is replaced for the reference."""
    wd = None if w is None else w.to(DEV)
    res = L.spec_lm_head_loss(h, wt, y.to(DEV), temperature=T, row_weight=wd, grad=True, **kw)
    only = L.spec_lm_head_loss(h, wt, y.to(DEV), temperature=T, row_weight=wd)
    torch.cuda.synchronize()
    out = (y < 0) | (y >= len(wt)) | (torch.zeros(len(y), dtype=torch.bool) if w is None else w == 0)
    bad = torch.isnan(h).any(dim=1).cpu()
    hc = torch.where((out & bad).to(DEV)[:, None], torch.zeros_like(h), h)
    ref = O.head(hc.double(), wt.double(), y, T, w)
    for o in (res, only):
        for k in ("loss", "log_z"):
            r, e = n64(ref[k]).copy(), n64(ref["e_" + k])
            if k == "loss":
                r[((y < 0) | (y >= len(wt))).numpy()] = 0.0
            unseen = (out & bad).numpy() if k == "log_z" else (bad & (w == 0)).numpy() if w is not None else np.zeros(len(y), bool)
            within(n64(o[k])[~unseen], r[~unseen], e[~unseen], k)
    for k in ("d_hidden", "d_weight"):
        r, e = ref[k], ref["e_" + k]
        off = (res[k].double() - r).abs() - (e + O.HALF[BF] * (r.abs() + e) + 2.0 ** -133)
        assert not torch.isnan(off).any(), k
        assert float(off.max()) <= 0, (k, float(off.max()), torch.nonzero(off == off.max())[0].tolist())
    assert "d_hidden" not in only and "d_weight" not in only
    return res


def head_of(R, V, D, seed, scale=1.3):
    g = torch.Generator().manual_seed(seed)
    wt = (torch.randn((V, D), generator=g) * (scale / D ** 0.5)).to(BF)
    y = torch.randint(0, V, (R,), generator=g)
    h = (torch.randn((R, D), generator=g) + 4.0 * wt[y].float() * torch.rand((R, 1), generator=g)).to(BF)
    return h.to(DEV), wt.to(DEV), y.to(torch.int32)


@pytest.mark.parametrize("R,V,D,T", [(1, 1, 8, 1.0), (1, 5, 8, 2.0), (3, 257, 24, 0.7), (64, 300, 72, 1.0), (65, 1000, 64, 1.0),
                                     (127, 511, 264, 0.5), (128, 513, 136, 1.0), (129, 700, 200, 1.0), (300, 4173, 192, 0.7),
                                     (515, 2000, 328, 2.0), (257, 9000, 520, 1.0)])
def test_head_loss_sizes(R, V, D, T):
    note(f"case head loss R={R} V={V} D={D} T={T}")
    h, wt, y = head_of(R, V, D, R + V + D)
    w = torch.from_numpy(np.random.default_rng(R).uniform(-0.5, 2, R).astype(np.float32))
    check_head(h, wt, y, T, w)


def test_head_loss_rows_left_out():
    """Targets outside the vocabulary and weights of zero: those rows give no gradient, also where
    their hidden states are NaN."""
    R, V, D = 200, 900, 96
    h, wt, y = head_of(R, V, D, 5)
    w = torch.ones(R)
    y[0], y[1], y[2], y[3] = -1, V, 2 ** 31 - 1, -2 ** 31
    w[4] = w[199] = 0.0
    h[0], h[4, 7], h[199] = np.nan, np.nan, np.nan
    res = check_head(h, wt, y, 1.0, w)
    assert (res["loss"][:4] == 0).all() and torch.isnan(res["loss"][4]) and torch.isnan(res["log_z"][0])
    assert (res["d_hidden"][:5] == 0).all() and (res["d_hidden"][199] == 0).all()
    check_head(*head_of(70, 300, 64, 6)[:2], torch.full((70,), -1, dtype=torch.int32), 1.0, None)   # none is left


def test_head_loss_nonfinite_rows():
    """A NaN or infinity in a row that counts: its loss is NaN, its neighbours' losses and hidden
    gradients are not touched."""
    R, V, D = 140, 700, 64
    h, wt, y = head_of(R, V, D, 8)
    clean = L.spec_lm_head_loss(h, wt, y.to(DEV), grad="hidden")
    h[3, 5], h[130, 0] = np.nan, np.inf
    res = L.spec_lm_head_loss(h, wt, y.to(DEV), grad="hidden")
    torch.cuda.synchronize()
    ok = torch.ones(R, dtype=torch.bool)
    ok[3] = ok[130] = False
    for k in ("loss", "log_z", "d_hidden"):
        assert torch.equal(res[k][ok], clean[k][ok]), k
        assert torch.isnan(res[k][~ok]).all(), k
    assert "d_weight" not in res
    wt[17] = -np.inf                                  # a token whose logits are NaN or infinite
    res = L.spec_lm_head_loss(h, wt, y.to(DEV))
    assert torch.isnan(res["loss"]).all()


def test_head_loss_strided_with_nan_padding():
    R, V, D, pad = 150, 900, 72, 24
    h, wt, y = head_of(R, V, D, 12)
    hb = torch.full((R, D + pad), float("nan"), dtype=BF, device=DEV)
    wb = torch.full((V, D + pad), float("nan"), dtype=BF, device=DEV)
    hb[:, 8:8 + D], wb[:, 16:16 + D] = h, wt
    dh = torch.full((R, D + 16), 7.0, dtype=BF, device=DEV)
    dw = torch.full((V + 2, D + 8), 7.0, dtype=BF, device=DEV)
    n = L.spec_lm_head_loss_workspace_bytes(R, V, D, True)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)     # NaN in every type
    check_head(hb[:, 8:8 + D], wb[:, 16:16 + D], y, 1.0, None, out={"d_hidden": dh[:, :D], "d_weight": dw[1:-1, 8:]}, workspace=ws)
    assert (dh[:, D:] == 7).all() and (dw[:, :8] == 7).all() and (dw[0] == 7).all() and (dw[-1] == 7).all()


@pytest.mark.parametrize("T", [0.01, 1e-30, 50.0])
def test_temperatures_far_from_one(T):
    """Sharp and flat distributions; at 1e-30 the distances alone stay in fp32's range."""
    T = float(np.float32(T))   # what the entry points take: 0.01 itself is 2e-8 off it, times log Z = 1500
    l = rows_of(4, 9000, BF, 31).to(DEV)
    check_topk(l, 20, T)
    index, t, lz = teacher_of(l, 20, T, 3, True) if T > 1e-3 else (*teacher_of(l, 20, 1.0, 3, False)[:2], None)
    if T > 1e-3:
        check_distill(l, index, t, lz, T, None)
    h, wt, y = head_of(70, 900, 64, 41)
    if T > 1e-3:
        check_head(h, wt, y, T, None)
    else:
        # one-hot at the largest logit: loss (max - l_y) / T, gradients of one token against another
        best = (h.double() @ wt.double().T).argmax(dim=1).int()
        w = torch.full((70,), T)
        res = L.spec_lm_head_loss(h, wt, best, temperature=T, row_weight=w.to(DEV), grad=True)
        other = (best + 1) % 900
        res2 = L.spec_lm_head_loss(h, wt, other, temperature=T, row_weight=w.to(DEV), grad="hidden")
        torch.cuda.synchronize()
        assert (res["d_hidden"] == 0).all() and (res["d_weight"] == 0).all()
        ref = wt[best.long()].double() - wt[other.long()].double()
        off = (res2["d_hidden"].double() - ref).abs() - (2 * O.U * wt.double().abs().sum(dim=0) + O.HALF[BF] * ref.abs())
        assert float(off.max()) <= 0


def test_offsets_past_32_bits():
    """More than 2^31 logits, and a head of more than 2^31 weights: the far ends are right."""
    R, V, K = 14200, 151936, 8
    note(f"case offsets R={R} V={V}")
    l = torch.zeros((R, V), dtype=BF, device=DEV)
    far = rows_of(3, V, BF, 5)
    l[-3:] = far.to(DEV)
    rec = L.spec_row_topk(l, K)
    index, logit, log_z = O.topk(n64(far), K, 1.0)
    np.testing.assert_array_equal(rec["index"][-3:].cpu().numpy(), index)
    np.testing.assert_array_equal(rec["index"][:2].cpu().numpy(), np.arange(K)[None].repeat(2, 0))
    i, t, lz = teacher_of(far, K, 1.0, 2, True)
    big = [v.new_zeros((R,) + tuple(v.shape[1:])) for v in (i, t, lz)]
    big[0].fill_(-1)
    for b, v in zip(big, (i, t, lz)):
        b[-3:] = v
    big = [b.to(DEV) for b in big]
    res = L.spec_topk_distill(l, big[0], big[1], teacher_log_z=big[2], grad=True, out={"d_logits": l})
    torch.cuda.synchronize()
    loss, _, d, e_loss, e_d = O.distill(n64(far), i.numpy(), t.numpy(), n64(lz), 1.0, None)
    within(n64(res["loss"][-3:]), loss, e_loss, "loss")
    within(n64(l[-3:]), d, e_d + O.HALF[BF] * (np.abs(d) + e_d), "d_logits")
    assert (res["loss"][:-3] == 0).all() and not l[:-3].any()
    del l, res, rec
    V, D = 1 << 21, 1032
    note(f"case offsets head V={V} D={D}")
    g = torch.Generator(device=DEV).manual_seed(1)
    wt = torch.empty((V, D), dtype=BF, device=DEV).normal_(0, 0.04, generator=g)
    h = torch.randn((3, D), generator=g, device=DEV).to(BF)
    y = torch.tensor([V - 1, 5, -1], dtype=torch.int32, device=DEV)
    res = L.spec_lm_head_loss(h, wt, y, grad=True)
    torch.cuda.synchronize()
    lz, dh = torch.full((3,), -np.inf, dtype=torch.float64, device=DEV), torch.zeros((3, D), dtype=torch.float64, device=DEV)
    for a in range(0, V, 1 << 18):
        lz = torch.logaddexp(lz, torch.logsumexp(h.double() @ wt[a:a + (1 << 18)].double().T, dim=1))
    ly = (h[:2].double() * wt[y[:2].long()].double()).sum(dim=1)
    delta = float(D * O.U * (h.double().abs().sum(dim=1) * 0.25).max())     # |w| < 0.25: six deviations
    assert (res["loss"][:2].double() - (lz[:2] - ly)).abs().max() <= 2 * delta + 2 * O.LZ + 4 * O.U * 20
    for a in range(0, V, 1 << 18):
        w = wt[a:a + (1 << 18)].double()
        p = torch.exp(h.double() @ w.T - lz[:, None])
        p[2] = 0.0
        dh += p @ w
        for r in (0, 1):
            if a <= int(y[r]) < a + (1 << 18):
                p[r, int(y[r]) - a] -= 1.0
        ref = p.T @ h.double()
        got = res["d_weight"][a:a + (1 << 18)].double()
        e = p.abs().T @ h.double().abs() * (2 * O.HALF[BF] + 2 * delta + 4 * O.LZ + 1e-4) + 2.0 ** -133
        assert float(((got - ref).abs() - e).max()) <= 0, a
    dh[:2] -= wt[y[:2].long()].double()
    dh[2] = 0.0
    # the probabilities' roundings to bf16 are spread over 2^21 tokens: their sum against |w| < 0.25
    assert float((res["d_hidden"].double() - dh).abs().max()) <= 0.25 * (O.HALF[BF] + 2 * delta + 1e-4) + O.HALF[BF] * float(dh.abs().max())


def test_head_loss_one_gradient_at_a_time_and_no_rows():
    h, wt, y = head_of(90, 1200, 128, 3)
    both = L.spec_lm_head_loss(h, wt, y.to(DEV), grad=True)
    a, b = (L.spec_lm_head_loss(h, wt, y.to(DEV), grad=g) for g in ("hidden", "weight"))
    torch.cuda.synchronize()
    assert "d_weight" not in a and "d_hidden" not in b
    assert torch.equal(a["d_hidden"], both["d_hidden"]) and torch.equal(b["d_weight"], both["d_weight"])
    none = L.spec_lm_head_loss(h[:0], wt, y[:0].to(DEV), grad=True)
    assert none["loss"].shape == (0,) and (none["d_weight"] == 0).all()


def test_head_loss_several_pieces_and_splits():
    """More logits than one piece holds, a ragged last piece, a hidden size of one tile and a bit."""
    R, V, D = 2100, 130001, 264
    note(f"case head loss in pieces R={R} V={V} D={D}")
    h, wt, y = head_of(R, V, D, 21)
    w = torch.full((R,), 1.0 / R)
    check_head(h, wt, y, 1.0, w)


def test_head_loss_formula_against_differences():
    """The definition's gradients against central differences of its loss, in 64 bits."""
    g = torch.Generator().manual_seed(2)
    h, wt = torch.randn((3, 8), generator=g).double(), torch.randn((11, 8), generator=g).double()
    y, w, T = torch.tensor([4, -1, 10]), torch.tensor([1.0, 3.0, -0.5]), 0.6
    ref = O.head(h, wt, y, T, w)
    total = lambda a, b: float((O.head(a, b, y, T, w)["loss"] * w.double()).sum())  # noqa: E731
    for name, x, grad in (("h", h, ref["d_hidden"]), ("w", wt, ref["d_weight"])):
        for i, j in ((0, 0), (1, 3), (2, 7)):
            e = torch.zeros_like(x)
            e[i, j] = 1e-5
            diff = (total(h + e, wt) - total(h - e, wt) if name == "h" else total(h, wt + e) - total(h, wt - e)) / 2e-5
            assert abs(diff - float(grad[i, j])) <= 1e-7


# ---------------------------------------------------------------- together, streams and graphs

def test_round_to_training_step():
    """A verification round and the step that learns from it: the target rows' records, distillation
    of the draft rows, the head's loss on the tokens that verification emitted."""
    inp = W.make_inputs(3, B=9, V=2 * 4096 + 72, seed=12)
    d = H.to_device(inp)
    G, B, V = int(inp.gammas.max()), 9, 2 * 4096 + 72
    ver = L.spec_verify_batch(d["target"], d["draft"], d["tokens"], d["cu"], G, temperature=0.7, seed=3, step=1)
    rec = check_topk(d["target"], 32, 0.7)
    cu = inp.cu_draft.astype(np.int64)
    rows = np.concatenate([np.arange(cu[b] + b, cu[b + 1] + b) for b in range(B)])      # target rows of the draft positions
    pick = torch.from_numpy(rows).to(DEV)
    idx, val, lz = rec["index"][pick].contiguous(), rec["logit"][pick].contiguous(), rec["log_z"][pick].contiguous()
    Rd = len(rows)
    w = torch.full((Rd,), 1.0 / Rd)
    res = check_distill(d["draft"], idx.cpu(), val.cpu(), lz.cpu(), 0.7, w)
    assert float(res["loss"].min()) > 0
    tok = ver["tokens"].reshape(-1)                                                     # -1 past each request's last token
    g = torch.Generator().manual_seed(4)
    h = torch.randn((len(tok), 64), generator=g).to(BF).to(DEV)
    wt = (torch.randn((V, 64), generator=g) * 0.2).to(BF).to(DEV)
    out = check_head(h, wt, tok.cpu(), 1.0, None)
    assert ((out["loss"] == 0) == (tok < 0)).all()


def _step(args, ws=None):
    l, s, h, wt, y = args
    kw = [{} if ws is None else {"workspace": x} for x in (ws or [None] * 3)]
    rec = L.spec_row_topk(l, 24, **kw[0])
    a = L.spec_topk_distill(s, rec["index"], rec["logit"], teacher_log_z=rec["log_z"], grad=True, **kw[1])
    b = L.spec_lm_head_loss(h, wt, y, grad=True, **kw[2])
    return [rec["index"], rec["logit"], rec["log_z"], a["loss"], a["d_logits"], b["loss"], b["d_hidden"], b["d_weight"]]


def _step_inputs(seed):
    h, wt, y = head_of(100, 3000, 128, seed)
    return [rows_of(20, 30000, BF, seed).to(DEV), rows_of(20, 30000, BF, seed + 1).to(DEV), h, wt, y.to(DEV)]


@pytest.mark.parametrize("own_workspaces", [True, False])
def test_graph_replays_match_eager(own_workspaces):
    """Two captured steps, replayed in turn with new inputs, eager calls and waits in between."""
    torch.cuda.synchronize()
    sizes = (L.spec_row_topk_workspace_bytes(20, 30000, 24), L.spec_topk_distill_workspace_bytes(20, 30000, 24, True),
             L.spec_lm_head_loss_workspace_bytes(100, 3000, 128, True))
    graphs = []
    for k in range(2):
        args = _step_inputs(40 + k)
        ws = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes] if own_workspaces else None
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            _step(args, ws)                    # first call of the kernels outside the capture
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = _step(args, ws)
        graphs.append((g, args, outs))
    for rep in range(4):
        for k in (rep % 2, 1 - rep % 2):
            g, args, outs = graphs[k]
            for dst, src in zip(args, _step_inputs(100 + 10 * rep + k)):
                dst.copy_(src)
            g.replay()
            eager = _step(_step_inputs(100 + 10 * rep + k))
            torch.cuda.synchronize()
            for i, (x, z) in enumerate(zip(outs, eager)):
                assert torch.equal(x, z), (rep, k, i)


def test_streams_side_by_side():
    """Calls without workspaces on several streams at once, the stream given or current."""
    args = [_step_inputs(60 + k) for k in range(3)]
    want = [_step(a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [None] * 3
    for _ in range(3):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k] = _step(args[k])
    torch.cuda.synchronize()
    for k in range(3):
        for i, (x, z) in enumerate(zip(got[k], want[k])):
            assert torch.equal(x, z), (k, i)
    rec = L.spec_row_topk(args[0][0], 24, stream=streams[1])
    torch.cuda.synchronize()
    assert torch.equal(rec["index"], want[0][0])


def test_outputs_repeat_bit_for_bit():
    args = _step_inputs(80)
    first = _step(args)
    for _ in range(3):
        for x, z in zip(_step(args), first):
            assert torch.equal(x, z)


def test_refusals_on_the_gpu():
    l = torch.zeros((4, 100), device=DEV)
    idx, t = torch.zeros((4, 3), dtype=torch.int32, device=DEV), torch.zeros((4, 3), device=DEV)
    h, wt = torch.zeros((4, 64), dtype=BF, device=DEV), torch.zeros((10, 64), dtype=BF, device=DEV)
    y = torch.zeros(4, dtype=torch.int32, device=DEV)
    with pytest.raises(TypeError):
        L.spec_row_topk(l.half(), 3)
    for k in (0, -1):
        with pytest.raises(ValueError):
            L.spec_row_topk(l, k)
    with pytest.raises(RuntimeError, match="-2"):
        L.spec_row_topk(l, 257)
    for T in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(RuntimeError, match="-1"):
            L.spec_row_topk(l, 3, temperature=T)
        with pytest.raises(RuntimeError, match="-1"):
            L.spec_topk_distill(l, idx, t, temperature=T)
        with pytest.raises(RuntimeError, match="-1"):
            L.spec_lm_head_loss(h, wt, y, temperature=T)
    with pytest.raises(ValueError):
        L.spec_row_topk(l.t(), 3)
    with pytest.raises(ValueError):
        L.spec_row_topk(l[:1].expand(4, 100), 3)
    with pytest.raises(ValueError):
        L.spec_row_topk(l, 3, out={"index": torch.zeros((4, 2), dtype=torch.int32, device=DEV)})
    with pytest.raises(ValueError):
        L.spec_row_topk(l, 3, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    for bad in ((idx.long(), t), (idx, t.double()), (idx[:3], t), (idx, t[:, :2]), (idx.cpu(), t)):
        with pytest.raises(ValueError):
            L.spec_topk_distill(l, *bad)
    with pytest.raises(ValueError):
        L.spec_topk_distill(l, idx, t, row_weight=torch.ones(3, device=DEV))
    with pytest.raises(ValueError):
        L.spec_topk_distill(l, idx, t, grad=True, out={"d_logits": l.to(BF)})
    with pytest.raises(ValueError):
        L.spec_lm_head_loss(h.float(), wt, y)
    with pytest.raises(ValueError):
        L.spec_lm_head_loss(h, wt[:, :32], y)
    with pytest.raises(ValueError):
        L.spec_lm_head_loss(h, wt, y.long())
    with pytest.raises(ValueError):
        L.spec_lm_head_loss(h, wt, y, grad="both")
    with pytest.raises(RuntimeError, match="-2"):
        L.spec_lm_head_loss(h[:, :60].contiguous(), wt[:, :60].contiguous(), y)
    with pytest.raises(RuntimeError, match="-1"):
        L.spec_lm_head_loss(h, wt, y, grad="hidden", out={"d_hidden": h})
    assert (h == 0).all() and (l == 0).all()
