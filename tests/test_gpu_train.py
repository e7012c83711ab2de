"""The training form's operators against plain implementations in 64 bits.

Tolerances follow from the arithmetic.  eps = 2^-24 is the rounding of one
fp32 operation, u the rounding of the output's type (bf16 2^-8, fp16 2^-11,
fp32 2^-24: half a spacing).  A sum of n terms by threads and then by shuffles
errs by at most (adds in the longest chain) * eps * sum|terms|; the chains are
at most cols / 1024 + 32 long within a row, and (rows / 64 + 64) long over
rows.  Each bound below is (chain + a few operations) * eps times the sum of the
magnitudes that enter, plus u times the result.
"""
import math

import pytest
import torch

import mxfp4_mixture_experts_02_gb300 as moe

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=FP, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(dtype)


def within(got, want, bound):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), "%d of %d past the bound, worst %.3g of it" % (
        int(bad.sum()), bad.numel(), float((err / bound.clamp_min(1e-300)).max()))


# ------------------------------------------------------------------ layer norm
NORM_SIZES = [(1, 1), (1, 64), (3, 7), (5, 33), (2, 1021), (33, 64), (130, 200), (7, 512), (32, 3584), (9, 3585),
              (64, 4096), (3, 4104), (5, 7168), (4, 8191), (2, 16384), (3, 20000), (2, 32771), (700, 1000), (1300, 24)]


def norm_ref(h, w, b, eps):
    h = h.double()
    mean = h.mean(1, keepdim=True)
    d = h - mean
    rstd = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + eps)
    y = d * rstd
    if w is not None:
        y = y * w.double()
    if b is not None:
        y = y + b.double()
    return y, mean, rstd


def check_norm(x, w, b, res, eps, y, h, mean, rstd):
    if res is not None:
        assert torch.equal(h, (x.float() + res.float()).to(x.dtype))
    else:
        assert h is x
    want, m, r = norm_ref(h, w, b, eps)
    k = (x.shape[1] / 1024 + 64) * EPS
    hd = h.double()
    dm = k * hd.abs().mean(1, keepdim=True) + TINY[FP]
    within(mean[:, None], m, dm)
    # a distance from the mean errs by the mean's error and one rounding; the
    # variance by twice that against the deviation, and its own sum
    var = (hd - m).pow(2).mean(1, keepdim=True)
    dev = dm + EPS * (hd - m).abs().amax(1, keepdim=True)
    dr = r * (k + 4 * EPS + 0.5 * (2 * dev * var.sqrt() + dev * dev) / (var + eps))
    within(rstd[:, None], r, dr)
    wd = w.double().abs() if w is not None else 1.0
    bd = b.double().abs() if b is not None else 0.0
    fp = wd * ((hd - m).abs() * (dr + 4 * EPS * r) + (dm + EPS * hd.abs()) * (r + dr)) + EPS * (want.abs() + bd)
    within(y, want, fp + U[x.dtype] * (want.abs() + fp) + TINY[x.dtype])


@pytest.mark.parametrize("rows,cols", NORM_SIZES)
@pytest.mark.parametrize("dtype,w_dtype", [(BF, BF), (BF, FP), (HF, HF), (FP, FP)])
def test_layer_norm(rows, cols, dtype, w_dtype):
    g = gen(rows * 100003 + cols)
    x = randn(g, rows, cols, dtype=dtype, scale=2.0, shift=0.5)
    w, b = randn(g, cols, dtype=w_dtype, scale=0.2, shift=1.0), randn(g, cols, dtype=w_dtype, scale=0.2)
    res = randn(g, rows, cols, dtype=dtype)
    for ww, bb, rr in ((w, b, None), (w, b, res), (None, None, res), (w, None, None), (None, b, None)):
        check_norm(x, ww, bb, rr, 1e-5, *moe.moe_layer_norm(x, ww, bb, rr))


def norm_grad_ref(dy, h, mean, rstd, w, dh):
    xh = (h.double() - mean.double()[:, None]) * rstd.double()[:, None]
    a = dy.double() * (w.double() if w is not None else 1.0)
    ax = (a * xh)
    dx = rstd.double()[:, None] * (a - a.mean(1, keepdim=True) - xh * ax.mean(1, keepdim=True))
    size = rstd.double()[:, None] * (a.abs() + a.abs().mean(1, keepdim=True) + xh.abs() * ax.abs().mean(1, keepdim=True))
    if dh is not None:
        dx, size = dx + dh.double(), size + dh.double().abs()
    return dx, size, (dy.double() * xh).sum(0), (dy.double() * xh).abs().sum(0), dy.double().sum(0), \
        dy.double().abs().sum(0)


def check_norm_grad(dy, h, mean, rstd, w, dh, dx, dw, db):
    want, size, dw_ref, dw_size, db_ref, db_size = norm_grad_ref(dy, h, mean, rstd, w, dh)
    rows, cols = h.shape
    fp = (cols / 1024 + 64) * EPS * size
    within(dx, want, fp + U[h.dtype] * (want.abs() + fp) + TINY[h.dtype])
    k = (rows / 64 + 64) * EPS
    if w is None:
        assert dw is None
    else:
        assert dw.dtype == FP
        within(dw, dw_ref, k * dw_size + TINY[FP])
    if db is not None:
        within(db, db_ref, k * db_size + TINY[FP])


@pytest.mark.parametrize("rows,cols", NORM_SIZES)
@pytest.mark.parametrize("dtype,w_dtype", [(BF, BF), (BF, FP), (HF, FP), (FP, FP)])
def test_layer_norm_backward(rows, cols, dtype, w_dtype):
    g = gen(rows * 7 + cols)
    h = randn(g, rows, cols, dtype=dtype, scale=2.0, shift=0.5)
    w = randn(g, cols, dtype=w_dtype, scale=0.2, shift=1.0)
    _, _, mean, rstd = moe.moe_layer_norm(h, w)
    dy, dh = randn(g, rows, cols, dtype=dtype), randn(g, rows, cols, dtype=dtype)
    for ww, dd, bias in ((w, None, True), (w, dh, True), (None, dh, True), (w, dh, False), (None, None, False)):
        dx, dw, db = moe.moe_layer_norm_backward(dy, h, mean, rstd, ww, dh=dd, bias_grad=bias)
        assert (db is not None) == bias
        check_norm_grad(dy, h, mean, rstd, ww, dd, dx, dw, db)


@pytest.mark.parametrize("rows,cols,dtype", [(5000, 3584, BF), (20001, 129, HF), (3000, 1024, FP)])
def test_layer_norm_many_rows_and_repeats(rows, cols, dtype):
    g = gen(rows)
    x = randn(g, rows, cols, dtype=dtype, scale=2.0, shift=0.5)
    w, b = randn(g, cols, scale=0.2, shift=1.0), randn(g, cols)
    dy = randn(g, rows, cols, dtype=dtype)
    y, h, mean, rstd = moe.moe_layer_norm(x, w, b)
    check_norm(x, w, b, None, 1e-5, y, h, mean, rstd)
    first = moe.moe_layer_norm_backward(dy, h, mean, rstd, w)
    check_norm_grad(dy, h, mean, rstd, w, None, *first)
    for a, c in zip(first, moe.moe_layer_norm_backward(dy, h, mean, rstd, w)):
        assert torch.equal(a, c)  # no atomics: the same bits


# rows wider than the ring's threads hold, more of them than CTAs, on the grid
# and off it, on either side of the kernels' limits (16384 columns in the
# gradient, 32768 of 16 bits and 16384 of 32 forward)
@pytest.mark.parametrize("rows,cols,dtype", [
    (1, 8200, BF), (333, 8200, BF), (309, 9001, BF), (160, 16384, HF), (157, 16392, BF), (155, 28672, BF),
    (40, 28680, BF), (159, 20001, HF), (3, 32761, HF), (40, 32768, BF), (305, 8196, FP), (200, 8193, FP),
    (155, 16384, FP), (40, 16388, FP), (5, 16381, FP)])
def test_layer_norm_wide_rows(rows, cols, dtype):
    g = gen(rows * 31 + cols)
    x = randn(g, rows, cols, dtype=dtype, scale=2.0, shift=0.5)
    w, b = randn(g, cols, scale=0.2, shift=1.0), randn(g, cols, scale=0.2)
    res, dy, dh = (randn(g, rows, cols, dtype=dtype) for _ in range(3))
    check_norm(x, w, b, None, 1e-5, *moe.moe_layer_norm(x, w, b))
    y, h, mean, rstd = moe.moe_layer_norm(x, w, b, res)
    check_norm(x, w, b, res, 1e-5, y, h, mean, rstd)
    for dd, bias in ((None, True), (dh, True), (dh, False)):
        got = moe.moe_layer_norm_backward(dy, h, mean, rstd, w, dh=dd, bias_grad=bias)
        check_norm_grad(dy, h, mean, rstd, w, dd, *got)
        for p, q in zip(got, moe.moe_layer_norm_backward(dy, h, mean, rstd, w, dh=dd, bias_grad=bias)):
            assert p is q or torch.equal(p, q)
    place = dy.clone()
    for p, q in zip(moe.moe_layer_norm_backward(place, h, mean, rstd, w, dh=dh, dx=place),
                    moe.moe_layer_norm_backward(dy, h, mean, rstd, w, dh=dh)):
        assert torch.equal(p, q)


def test_layer_norm_gradient_matches_differences():
    g = gen(3)
    rows, cols, eps = 3, 10, 1e-3
    x, w, b = randn(g, rows, cols), randn(g, cols), randn(g, cols)
    out = randn(g, rows, cols)  # loss = <out, y> + <dh, h>
    dh = randn(g, rows, cols)
    _, h, mean, rstd = moe.moe_layer_norm(x, w, b, eps=eps)
    dx, dw, db = moe.moe_layer_norm_backward(out, h, mean, rstd, w, dh=dh)

    def loss(x, w, b):
        return ((norm_ref(x, w, b, eps)[0] * out.double()).sum() + (x * dh.double()).sum()).item()

    step = 1e-5
    for t, grad in ((x, dx), (w, dw), (b, db)):
        base = [x.double(), w.double(), b.double()]
        at = [i for i, s in enumerate((x, w, b)) if s is t][0]
        for i in range(t.numel()):
            v = []
            for sign in (1, -1):
                moved = [a.clone() for a in base]
                moved[at].view(-1)[i] += sign * step
                v.append(loss(*moved))
            # central differences in 64 bits err by about step^2 here, fp32 statistics by 1e-5
            assert abs((v[0] - v[1]) / (2 * step) - grad.view(-1)[i].item()) <= 2e-4


def test_layer_norm_in_place_and_misaligned():
    g = gen(11)
    for cols in (512, 20000):
        x, r = randn(g, 6, cols, dtype=BF), randn(g, 6, cols, dtype=BF)
        w = randn(g, cols, dtype=BF, shift=1.0)
        y, h, mean, rstd = moe.moe_layer_norm(x, w, None, r)
        for over in (x.clone(), r.clone()):  # h takes x's or the residual's place
            a, c = (over, r) if over is not x and torch.equal(over, x) else (x, over)
            y2, h2, _, _ = moe.moe_layer_norm(a, w, None, c, h=over)
            assert torch.equal(y, y2) and torch.equal(h, h2)
        dy, dh = randn(g, 6, cols, dtype=BF), randn(g, 6, cols, dtype=BF)
        want = moe.moe_layer_norm_backward(dy, h, mean, rstd, w, dh=dh)
        for name in ("dy", "dh"):
            ops = {"dy": dy.clone(), "dh": dh.clone()}
            got = moe.moe_layer_norm_backward(ops["dy"], h, mean, rstd, w, dh=ops["dh"], dx=ops[name])
            assert all(torch.equal(p, q) for p, q in zip(want, got))
        # rows that start one element past a 16-byte boundary
        xm = torch.empty(6 * cols + 1, dtype=BF, device="cuda")[1:].view(6, cols)
        xm.copy_(x)
        y3, h3, m3, r3 = moe.moe_layer_norm(xm, w, None, r)
        check_norm(xm, w, None, r, 1e-5, y3, h3, m3, r3)


def test_layer_norm_extreme_rows():
    x = torch.zeros(6, 96, device="cuda")
    x[1] = 7.25                      # no variance: the bias is left
    x[2] = 1e18                      # constant and large
    x[3, 5] = float("inf")
    x[4, 6] = float("nan")
    x[5] = 1e4 + torch.arange(96, device="cuda") / 64.0  # a mean far above the deviation
    b = torch.linspace(-1, 1, 96, device="cuda")
    y, _, mean, rstd = moe.moe_layer_norm(x, None, b, eps=1e-5)
    assert torch.equal(y[:3], b.expand(3, -1)) and torch.equal(mean[:3], torch.tensor([0, 7.25, 1e18], device="cuda"))
    assert torch.isnan(y[3]).all() and torch.isnan(y[4]).all()
    want, _, _ = norm_ref(x[5:], None, b, 1e-5)
    assert float((y[5:].double() - want).abs().max()) <= 96 * EPS * 1e4 / 0.43 + 1e-6


def test_layer_norm_no_rows():
    w = torch.ones(40, device="cuda", dtype=BF)
    x = torch.empty(0, 40, device="cuda", dtype=BF)
    y, h, mean, rstd = moe.moe_layer_norm(x, w, w)
    assert y.shape == (0, 40) and mean.shape == (0,)
    dx, dw, db = moe.moe_layer_norm_backward(x, x, mean, rstd, w)
    assert dx.shape == (0, 40) and not dw.any() and not db.any()


# ------------------------------------------------------------------ tokens <-> rows
#            T, E_global, E_local, offset, top_k, shared, hidden
TOKEN_CASES = [(1, 8, 8, 0, 1, 0, 1), (4, 8, 8, 0, 2, 0, 512), (7, 60, 15, 30, 4, 1, 33), (32, 896, 896, 0, 16, 0, 3584),
               (65, 896, 448, 448, 16, 1, 1000), (513, 64, 16, 48, 8, 0, 264), (300, 1024, 1023, 1, 32, 1, 72),
               (1100, 896, 896, 0, 16, 0, 130), (3, 16, 1, 15, 3, 0, 8200), (129, 5, 5, 0, 5, 1, 2049)]


def token_case(T, Eg, El, off, k, S, H, seed=0):
    g = gen(T + Eg + H + seed)
    shape = moe.MoeTokenShape(T, Eg, El, off, k, S, H)
    ids = torch.rand((T, Eg), generator=g, device="cuda").argsort(1)[:, :k].int()
    if S:
        ids = torch.cat([ids, torch.full((T, 1), Eg, device="cuda", dtype=torch.int32)], 1)
    w = torch.rand((T, k + S), generator=g, device="cuda")
    return g, shape, ids.contiguous(), w


def map_ref(shape, ids):
    flat = ids.reshape(-1).tolist()
    El, Et = shape.E_local, shape.E_local + shape.num_shared
    rows = [[] for _ in range(Et)]
    for s, e in enumerate(flat):
        if shape.expert_offset <= e < shape.expert_offset + El:
            rows[e - shape.expert_offset].append(s)
        elif shape.E_global <= e < shape.E_global + shape.num_shared:
            rows[El + e - shape.E_global].append(s)
    a = [s for r in rows for s in r]
    c = [-1] * len(flat)
    for i, s in enumerate(a):
        c[s] = i
    off = [0]
    for r in rows:
        off.append(off[-1] + len(r))
    return a, c, off


@pytest.mark.parametrize("case", TOKEN_CASES)
def test_token_map(case):
    _, shape, ids, _ = token_case(*case)
    a, c, off = map_ref(shape, ids)
    maps = moe.moe_token_map(shape, ids)
    assert maps.expert_offsets.tolist() == off
    assert maps.c_map.view(-1).tolist() == c
    assert maps.a_map[:len(a)].tolist() == a


def test_token_map_repeated_and_foreign_ids():
    shape = moe.MoeTokenShape(3, 8, 4, 2, 4, 0, 16)
    ids = torch.tensor([[2, 2, 9, -1], [5, 6, 1, 2], [0, 1, 7, 6]], dtype=torch.int32, device="cuda")
    a, c, off = map_ref(shape, ids)
    maps = moe.moe_token_map(shape, ids)
    assert (maps.expert_offsets.tolist(), maps.c_map.view(-1).tolist(), maps.a_map[:len(a)].tolist()) == (off, c, a)


def test_token_map_long_batch_and_given_buffers():
    _, shape, ids, _ = token_case(5000, 896, 448, 0, 16, 0, 8)
    maps = moe.MoeTokenMap(torch.full((80000,), -7, dtype=torch.int32, device="cuda"),
                           torch.empty((5000, 16), dtype=torch.int32, device="cuda"),
                           torch.empty(449, dtype=torch.int32, device="cuda"))
    got = moe.moe_token_map(shape, ids, ws=moe.token_map_workspace(shape), maps=maps)
    a, c, off = map_ref(shape, ids)
    assert got is maps and maps.expert_offsets.tolist() == off and maps.c_map.view(-1).tolist() == c
    assert maps.a_map[:len(a)].tolist() == a and (maps.a_map[len(a):] == -7).all()


@pytest.mark.parametrize("T", [1, 127, 128, 129, 2047, 2048, 2049, 20000, 65536, 65537])
@pytest.mark.parametrize("E,local", [(32, 32), (1024, 512)])
def test_token_map_on_either_side_of_each_way_of_sorting(T, E, local):
    # 16 slots a token: 2048, 32768 and 1048576 slots are where the launches change
    g = gen(T)
    shape = moe.MoeTokenShape(T, E, local, E - local, 16, 0, 8)
    ids = torch.randint(0, E, (T, 16), generator=g, device="cuda", dtype=torch.int32)
    maps = moe.moe_token_map(shape, ids)
    e = ids.view(-1).long() - (E - local)
    e = torch.where(e >= 0, e, local)
    by, order = torch.sort(e, stable=True)
    R = int((by < local).sum())
    c = torch.full_like(order, -1)
    c[order[:R]] = torch.arange(R, device="cuda")
    assert torch.equal(maps.a_map[:R].long(), order[:R]) and torch.equal(maps.c_map.view(-1).long(), c)
    assert torch.equal(maps.expert_offsets.long(), torch.searchsorted(by, torch.arange(local + 1, device="cuda")))


def gather(rows, c):
    """[T, k', H] in 64 bits, zero without a row."""
    return torch.where((c >= 0)[:, :, None], rows[c.clamp_min(0).long()].double(), 0.0)


@pytest.mark.parametrize("case", TOKEN_CASES)
@pytest.mark.parametrize("dtype", [BF, HF, FP])
def test_permute_and_unpermute(case, dtype):
    g, shape, ids, w = token_case(*case)
    T, H, kp = shape.T, shape.hidden, shape.kp
    maps = moe.moe_token_map(shape, ids)
    c = maps.c_map
    R = int(maps.expert_offsets[-1])
    x = randn(g, T, H, dtype=dtype)
    rows = torch.full((T * kp, H), -3.0, dtype=dtype, device="cuda")
    assert moe.moe_permute(shape, x, maps, rows=rows) is rows
    assert torch.equal(rows[:R], x[maps.a_map[:R].long() // kp]) and (rows[R:] == -3.0).all()

    # rows past R are never read: NaN there does not show
    y = randn(g, T * kp, H, dtype=dtype)
    y[R:] = float("nan")
    terms = gather(y, c) * w.double()[:, :, None]
    fp = (kp + 2) * EPS * terms.abs().sum(1)
    want = terms.sum(1)
    within(moe.moe_unpermute(shape, y, w, maps), want, fp + U[dtype] * (want.abs() + fp) + TINY[dtype])
    terms = gather(y, c)
    fp, want = (kp + 2) * EPS * terms.abs().sum(1), terms.sum(1)
    within(moe.moe_permute_backward(shape, y, maps), want, fp + U[dtype] * (want.abs() + fp) + TINY[dtype])

    dout = randn(g, T, H, dtype=dtype)
    dy = torch.full_like(y, -3.0)
    got, dw = moe.moe_unpermute_backward(shape, dout, y, w, maps, dy=dy)
    prods = gather(y, c) * dout.double()[:, None, :]
    within(dw, prods.sum(2), (H / 128 + 32) * EPS * prods.abs().sum(2))
    assert got is dy and (dy[R:] == -3.0).all() and not dw[c < 0].any()
    slot = maps.a_map[:R].long()
    want = dout[slot // kp].double() * w.view(-1)[slot].double()[:, None]
    within(dy[:R], want, (EPS + U[dtype]) * want.abs() + TINY[dtype])
    # over the rows themselves
    dw2 = moe.moe_unpermute_backward(shape, dout, y, w, maps, dy=y)[1]
    assert torch.equal(y[:R], dy[:R]) and torch.equal(dw2, dw)


def test_tokens_without_any_row():
    # all picks elsewhere: zeros come back, nothing is written
    shape = moe.MoeTokenShape(9, 16, 4, 12, 2, 0, 40)
    ids = torch.zeros((9, 2), dtype=torch.int32, device="cuda") + torch.arange(2, device="cuda", dtype=torch.int32)
    maps = moe.moe_token_map(shape, ids)
    assert not maps.expert_offsets.any() and (maps.c_map == -1).all()
    rows = torch.full((18, 40), float("nan"), device="cuda")
    w = torch.full((9, 2), float("inf"), device="cuda")
    assert not moe.moe_unpermute(shape, rows, w, maps).any()
    assert not moe.moe_permute_backward(shape, rows, maps).any()
    dy, dw = moe.moe_unpermute_backward(shape, torch.ones(9, 40, device="cuda"), rows, w, maps,
                                        dy=torch.ones_like(rows))
    assert (dy == 1).all() and not dw.any()
    assert (moe.moe_permute(shape, torch.ones(9, 40, device="cuda"), maps, rows=torch.zeros_like(rows)) == 0).all()


def test_tokens_no_tokens():
    shape = moe.MoeTokenShape(0, 16, 16, 0, 2, 0, 40)
    maps = moe.moe_token_map(shape, torch.empty((0, 2), dtype=torch.int32, device="cuda"))
    assert maps.expert_offsets.tolist() == [0] * 17
    x = torch.empty((0, 40), device="cuda")
    w = torch.empty((0, 2), device="cuda")
    assert moe.moe_permute(shape, x, maps).shape == (0, 40)
    assert moe.moe_unpermute(shape, x, w, maps).shape == (0, 40)
    assert moe.moe_permute_backward(shape, x, maps).shape == (0, 40)
    assert moe.moe_unpermute_backward(shape, x, x, w, maps)[1].shape == (0, 2)


def test_tokens_offsets_past_32_bits():
    # 8.6 GB of rows: row offsets pass 2^31 elements and 2^32 bytes
    T, k, H = 37450, 16, 7168
    shape = moe.MoeTokenShape(T, 64, 64, 0, k, 0, H)
    g = gen(5)
    ids = torch.rand((T, 64), generator=g, device="cuda").argsort(1)[:, :k].int().contiguous()
    w = torch.rand((T, k), generator=g, device="cuda")
    maps = moe.moe_token_map(shape, ids)
    assert T * k * H > 1 << 32
    x = randn(g, T, H, dtype=BF)
    rows = moe.moe_permute(shape, x, maps)
    at = torch.tensor([0, 1, T * k // 2, T * k - 2, T * k - 1], device="cuda")
    assert torch.equal(rows[at], x[maps.a_map[at].long() // k])
    out = moe.moe_unpermute(shape, rows, w, maps)
    t = torch.tensor([0, 7, T - 1], device="cuda")
    want = x[t].double() * w[t].double().sum(1, keepdim=True)
    within(out[t], want, (2 * k * EPS + 2 ** -8) * want.abs() * 1.01)
    dy, dw = moe.moe_unpermute_backward(shape, x, rows, w, maps, dy=rows)
    slot = maps.a_map[at].long()
    want = x[slot // k].double() * w.view(-1)[slot].double()[:, None]
    within(dy[at], want, (EPS + 2 ** -8) * want.abs())
    sq = x[t].double().pow(2).sum(1, keepdim=True)
    within(dw[t], sq.expand(-1, k), (H / 128 + 32) * EPS * sq.expand(-1, k))


def test_unpermute_gradient_matches_differences():
    g, shape, ids, w = token_case(5, 8, 4, 2, 3, 1, 6)
    maps = moe.moe_token_map(shape, ids)
    y, out = randn(g, 20, 6), randn(g, 5, 6)
    x = randn(g, 5, 6)
    dy, dw = moe.moe_unpermute_backward(shape, out, y, w, maps, dy=torch.zeros_like(y))
    step = 1e-4

    def loss(y, w):
        return ((gather(y, maps.c_map) * w[:, :, None]).sum(1) * out.double()).sum().item()

    for which, t, grad in ((0, y, dy), (1, w, dw)):
        for i in range(t.numel()):
            v = []
            for sign in (1, -1):
                ops = [y.double(), w.double()]
                ops[which] = ops[which].clone()
                ops[which].view(-1)[i] += sign * step
                v.append(loss(*ops))
            assert abs((v[0] - v[1]) / (2 * step) - grad.view(-1)[i].item()) <= 1e-5
    # permute: <drows, permute(x)> = <dx, x>
    rows = moe.moe_permute(shape, x, maps, rows=torch.zeros_like(y))
    R = int(maps.expert_offsets[-1])
    dx = moe.moe_permute_backward(shape, y, maps)
    a, b = (rows[:R].double() * y[:R].double()).sum().item(), (dx.double() * x.double()).sum().item()
    assert abs(a - b) <= 1e-5 * (1 + abs(a))


# ------------------------------------------------------------------ routing gradient
@pytest.mark.parametrize("T,E,k,S", [(1, 2, 1, 0), (3, 8, 8, 1), (5, 127, 4, 0), (33, 896, 16, 1), (1000, 60, 6, 0),
                                     (20000, 1024, 32, 1), (8, 1, 1, 1)])
def test_route_backward(T, E, k, S):
    g = gen(T + E)
    shape = moe.MoeTokenShape(T, E, E, 0, k, S, 512)
    logits, z = randn(g, T, E, scale=3.0), randn(g, T, 1, dtype=BF, scale=4.0) if S else None
    # moe_route's own picks and weights
    full = moe.MoeShape(T, T, E, min(E, 1024 - S), 0, k, S, 512, 128, 16, shared_scale=0.5)
    ids, w = moe.moe_route(full, logits, z)
    dw = randn(g, T, k + S)
    dl, dz = moe.moe_route_backward(shape, ids, w, dw, z, 0.5)
    wd, d = w[:, :k].double(), dw[:, :k].double()
    picked = wd * (d - (wd * d).sum(1, keepdim=True))
    want = torch.zeros(T, E, device="cuda", dtype=torch.float64).scatter_(1, ids[:, :k].long(), picked)
    size = torch.zeros_like(want).scatter_(1, ids[:, :k].long(), wd * (d.abs() + (wd * d).abs().sum(1, keepdim=True)))
    within(dl, want, 12 * EPS * size + TINY[FP])
    assert (dz is None) == (S == 0)
    if S:
        a = torch.sigmoid(z.double())
        want = dw[:, k:].double() * 0.5 * a * (1 - a)
        # expf within 2 units in the last place, the rest rounded once each; 1 - a to eps
        within(dz, want, 16 * EPS * (want.abs() + (dw[:, k:].double() * 0.5).abs() * a))


def test_route_backward_matches_differences():
    g = gen(9)
    T, E, k = 4, 9, 3
    shape = moe.MoeTokenShape(T, E, E, 0, k, 1, 512)
    full = moe.MoeShape(T, T, E, E, 0, k, 1, 512, 128, 16, shared_scale=0.25)
    logits, z, dw = randn(g, T, E), randn(g, T, 1, dtype=BF), randn(g, T, k + 1)
    ids, w = moe.moe_route(full, logits, z)
    dl, dz = moe.moe_route_backward(shape, ids, w, dw, z, 0.25)

    def loss(l, zz):
        p = torch.softmax(l.gather(1, ids[:, :k].long()), 1)
        return ((p * dw[:, :k].double()).sum() + (0.25 * torch.sigmoid(zz) * dw[:, k:].double()).sum()).item()

    step = 1e-5
    for which, grad in ((0, dl), (1, dz)):
        for i in range(grad.numel()):
            v = []
            for sign in (1, -1):
                ops = [logits.double(), z.double()]
                ops[which].view(-1)[i] += sign * step
                v.append(loss(*ops))
            assert abs((v[0] - v[1]) / (2 * step) - grad.view(-1)[i].item()) <= 1e-6


# ------------------------------------------------------------------ AdamW
HYPER = dict(lr=3e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)


def adamw_ref(p, g, m, v, step, scale, lr, betas, eps, weight_decay):
    g = g.double() * scale
    m = betas[0] * m + (1 - betas[0]) * g
    v = betas[1] * v + (1 - betas[1]) * g * g
    upd = lr * (m / (1 - betas[0] ** step)) / ((v / (1 - betas[1] ** step)).sqrt() + eps)
    return p.double() * (1 - lr * weight_decay) - upd, m, v, upd


SIZES = [1, 7, 31, 32, 33, 4095, 4096, 4097, 100003, 0, 512 * 128]


@pytest.mark.parametrize("g_dtype", [FP, BF, HF])
@pytest.mark.parametrize("scale", [None, 0.37])
def test_adamw_f32(g_dtype, scale):
    g = gen(1)
    ps = [randn(g, n, scale=0.1) for n in SIZES]
    gs = [torch.zeros(n, dtype=g_dtype, device="cuda") for n in SIZES]
    h = moe.adamw_tensors(ps, gs)
    c = None if scale is None else torch.tensor([scale], device="cuda")
    sc = 1.0 if scale is None else c.double().item()
    for step in (1, 2, 3):
        for t in gs:
            t.copy_(randn(g, t.numel(), scale=1e-2))
        before = [(p.clone(), m.double(), v.double()) for p, m, v in zip(h.params, h.m, h.v)]
        moe.moe_adamw(h, step, grad_scale=c, **HYPER)
        for (p0, m0, v0), p, gr, m, v in zip(before, h.params, h.grads, h.m, h.v):
            want, wm, wv, upd = adamw_ref(p0, gr, m0, v0, step, sc, **HYPER)
            gd = (gr.double() * sc).abs()
            # constants and operations each rounded once
            mb = 6 * EPS * (m0.abs() + gd)
            vb = 8 * EPS * (v0 + gd * gd)
            within(m, wm, mb + TINY[FP])
            within(v, wv, vb + TINY[FP])
            den = (wv / (1 - 0.999 ** step)).sqrt() + 1e-8
            rel = 0.5 * vb / wv.clamp_min(1e-300) + 8 * EPS
            within(p, want, 4 * EPS * p0.double().abs() + upd.abs() * rel + 2 * HYPER["lr"] * mb / den)


def mx_decode(codes, scales):
    n = codes.numel()
    s = torch.exp2(scales.double() - 127).repeat_interleave(32)[:n]
    return codes.view(torch.float8_e4m3fn).double() * s


def random_halves(seed, counter, n):
    """The 32 random bits of elements counter .. counter + n - 1 (Python integers)."""
    mask = (1 << 64) - 1
    out = []
    for c in range(counter, counter + n):
        z = (seed + (c // 2 + 1) * 0x9E3779B97F4A7C15) & mask
        z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & mask
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & mask
        z ^= z >> 31
        out.append((z >> (32 * (c & 1))) & 0xFFFFFFFF)
    return torch.tensor(out, dtype=torch.int64, device="cuda")


def check_mx(codes, scales, value, err, rand16, root):
    """Scale and codes of `value` (64 bits, known to the kernel to within `err`) by the format's rule.  A value whose
    error reaches a boundary (and 2^-28 from the move past the small codes) may fall on either side."""
    n = value.numel()
    pad = (-n) % 32
    blocks = torch.cat([value, value.new_zeros(pad)]).view(-1, 32)
    top = blocks.abs().amax(1)
    fl = torch.floor(torch.log2(top.clamp_min(1e-300)))
    e = torch.where(top > 0, fl - 7, torch.full_like(fl, -126)).clamp(-126, 126)
    got_e = scales.double() - 127
    near = (torch.log2(top.clamp_min(1e-300)) - torch.round(torch.log2(top.clamp_min(1e-300)))).abs() < 64 * EPS
    assert ((got_e == e) | (near & ((got_e - e).abs() <= 1))).all()
    q = value / torch.exp2(got_e).repeat_interleave(32)[:n]
    a = q.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))) - 3)
    pos = a / step + rand16.double() / 65536
    want = torch.floor(pos) * step
    if root:
        want = torch.where(value != 0, want.clamp_min(2.0 ** -9), want)
    got = codes.view(torch.float8_e4m3fn).double()
    tol = (err / torch.exp2(got_e).repeat_interleave(32)[:n] + 2.0 ** -28) / step + 1e-12  # in codes
    edge = (pos - torch.round(pos)).abs() <= tol
    diff = (got.abs() - want).abs()
    assert ((diff == 0) | (edge & (diff <= 2 * step))).all(), int(((diff != 0) & ~edge).sum())
    assert (diff != 0).double().mean() < 1e-3
    assert ((got == 0) | (torch.sign(got) == torch.sign(value))).all()


@pytest.mark.parametrize("g_dtype", [FP, BF, HF])
def test_adamw_mxfp8(g_dtype):
    sizes = [1, 7, 31, 32, 33, 4097, 0, 20000]
    g = gen(2)
    ps = [randn(g, n, scale=0.1) for n in sizes]
    gs = [torch.zeros(n, dtype=g_dtype, device="cuda") for n in sizes]
    h = moe.adamw_tensors(ps, gs, mxfp8=True)
    for step in (1, 2, 3):
        for i, t in enumerate(gs):
            # magnitudes over several decades within a block; one tensor with dead blocks
            t.copy_(randn(g, t.numel()) * torch.exp(3 * randn(g, t.numel()) - 6))
            if i == 5:
                t[64:1000] = 0
        old = [(p.clone(), mx_decode(m, ms), mx_decode(v, vs)) for p, m, ms, v, vs in
               zip(h.params, h.m, h.m_scale, h.v, h.v_scale)]
        moe.moe_adamw(h, step, seed=1000 + step, **HYPER)
        counter = 0
        for i, (p0, m0, r0) in enumerate(old):
            n = p0.numel()
            if n == 0:
                continue
            want, wm, wv, upd = adamw_ref(p0, gs[i], m0, r0 * r0, step, 1.0, **HYPER)
            gd = gs[i].double().abs()
            mb, vb = 6 * EPS * (m0.abs() + gd), 8 * EPS * (r0 * r0 + gd * gd)
            den = (wv / (1 - 0.999 ** step)).sqrt() + 1e-8
            rel = 0.5 * vb / wv.clamp_min(1e-300) + 8 * EPS
            within(h.params[i], want, 4 * EPS * p0.double().abs() + upd.abs() * rel + 2 * HYPER["lr"] * mb / den
                   + 1e-30)
            bits = random_halves(1000 + step, counter, n)
            check_mx(h.m[i], h.m_scale[i], wm, mb, bits & 0xFFFF, False)
            check_mx(h.v[i], h.v_scale[i], wv.sqrt(), wv.sqrt() * rel, bits >> 16, True)
            counter += (n + 31) // 32 * 32


def test_adamw_mxfp8_second_moment_follows_small_changes():
    # the gradient doubles: under rounding to nearest sqrt(v) would stay where it was (a step moves it by 0.15 %, a
    # code is 6 to 12 %); its mean has to follow v = v0 + (4 - 1)(1 - b2^s) to within a few standard errors
    n, steps = 1 << 16, 200
    p, gr = torch.zeros(n, device="cuda"), torch.full((n,), 1.0, device="cuda")
    h = moe.adamw_tensors([p], [gr], mxfp8=True)
    h.v[0].copy_(torch.full((n,), 128.0, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8))
    h.v_scale[0].fill_(127 - 7)  # sqrt(v) = 1
    gr.fill_(2.0)
    for s in range(steps):
        moe.moe_adamw(h, 1000 + s, lr=0.0, seed=12345 + s)
    v = mx_decode(h.v[0], h.v_scale[0]).pow(2).mean().item()
    want = 1 + 3 * (1 - 0.999 ** steps)
    # sqrt(v) is kept unbiased; its square carries the codes' variance (at most (1/8)^2 / 4 of it) on top
    assert want * 0.97 <= v <= want * 1.03


def test_adamw_more_tensors_than_a_launch_takes_and_misaligned():
    g = gen(4)
    sizes = [17 + 5 * (i % 40) for i in range(1000)]
    flat = [torch.empty(sum(sizes) + 1, device="cuda")[1:] for _ in range(2)]
    starts = [sum(sizes[:i]) for i in range(1000)]
    for mx in (False, True):
        flat[0].copy_(randn(g, sum(sizes)))
        flat[1].copy_(randn(g, sum(sizes)))
        ps, gs = ([f[b:b + n] for b, n in zip(starts, sizes)] for f in flat)
        before = flat[0].clone()
        h = moe.adamw_tensors(ps, gs, mxfp8=mx)
        moe.moe_adamw(h, 1, **HYPER)
        zero = torch.zeros_like(before).double()
        want, _, _, upd = adamw_ref(before, flat[1], zero, zero, 1, 1.0, **HYPER)
        within(flat[0], want, 4 * EPS * before.double().abs() + 40 * EPS * upd.abs())


@pytest.mark.parametrize("g_dtype", [BF, FP])
def test_adamw_mxfp8_long_tensors_and_scales_anywhere(g_dtype):
    """Work items of eight steps, the last of a tensor shorter, and scales off the 4-byte grid."""
    g = gen(7)
    sizes = [8 * 2048 * 152 * 32 + 5 * 2048 + 77, 3 * 2048 + 40, 70001]
    ps = [randn(g, n, scale=0.1) for n in sizes]
    gs = [(randn(g, n) * torch.exp(3 * randn(g, n) - 6)).to(g_dtype) for n in sizes]
    h = moe.adamw_tensors([p.clone() for p in ps], gs, mxfp8=True)
    blocks = [(n + 31) // 32 for n in sizes]
    flat = torch.zeros(sum(blocks) * 2 + 3, dtype=torch.uint8, device="cuda")
    cuts = torch.split(flat[3:], blocks * 2)
    odd = moe.MoeAdamwTensors([p.clone() for p in ps], gs, [torch.zeros_like(m) for m in h.m],
                              [torch.zeros_like(v) for v in h.v], list(cuts[:3]), list(cuts[3:]))
    for step in (1, 2):
        old = [(p.clone(), mx_decode(m, ms), mx_decode(v, vs)) for p, m, ms, v, vs in
               zip(h.params[1:], h.m[1:], h.m_scale[1:], h.v[1:], h.v_scale[1:])]
        some = [0, 2048 * 8 - 64, 2048 * 8 * 1000 + 32 * 301, sizes[0] // 32 * 32 - 4096]
        old += [(h.params[0][c:c + 4096].clone(), mx_decode(h.m[0][c:c + 4096], h.m_scale[0][c // 32:c // 32 + 128]),
                 mx_decode(h.v[0][c:c + 4096], h.v_scale[0][c // 32:c // 32 + 128])) for c in some]
        for t in (h, odd):
            moe.moe_adamw(t, step, seed=step, **HYPER)
        for name in ("params", "m", "v", "m_scale", "v_scale"):
            assert all(torch.equal(p, q) for p, q in zip(getattr(h, name), getattr(odd, name))), name
        first = (sizes[0] + 31) // 32 * 32
        second = first + (sizes[1] + 31) // 32 * 32
        at = [(1, 0, sizes[1], first), (2, 0, sizes[2], second)] + [(0, c, c + 4096, c) for c in some]
        for (p0, m0, r0), (i, lo, hi, counter) in zip(old, at):
            gr, b = gs[i][lo:hi], slice(lo // 32, (hi + 31) // 32)
            want, wm, wv, upd = adamw_ref(p0, gr, m0, r0 * r0, step, 1.0, **HYPER)
            gd = gr.double().abs()
            mb, vb = 6 * EPS * (m0.abs() + gd), 8 * EPS * (r0 * r0 + gd * gd)
            den = (wv / (1 - 0.999 ** step)).sqrt() + 1e-8
            rel = 0.5 * vb / wv.clamp_min(1e-300) + 8 * EPS
            within(h.params[i][lo:hi], want, 4 * EPS * p0.double().abs() + upd.abs() * rel
                   + 2 * HYPER["lr"] * mb / den + 1e-30)
            bits = random_halves(step, counter, hi - lo)
            check_mx(h.m[i][lo:hi], h.m_scale[i][b], wm, mb, bits & 0xFFFF, False)
            check_mx(h.v[i][lo:hi], h.v_scale[i][b], wv.sqrt(), wv.sqrt() * rel, bits >> 16, True)


def test_adamw_mxfp8_non_finite_in_whole_steps():
    n, at = 3 * 2048, (0, 2047, 2048 + 777)
    p, gr = torch.ones(n, device="cuda"), randn(gen(8), n)
    clean = moe.adamw_tensors([p.clone()], [gr.clone()], mxfp8=True)
    gr[list(at)] = torch.tensor([float("nan"), float("inf"), float("-inf")], device="cuda")
    h = moe.adamw_tensors([p], [gr], mxfp8=True)
    for t in (clean, h):
        moe.moe_adamw(t, 1, seed=3, **HYPER)
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    bad[list(at)] = True
    for t, s in (("m", "m_scale"), ("v", "v_scale")):
        got = mx_decode(getattr(h, t)[0], getattr(h, s)[0])
        assert torch.equal(torch.isnan(got), bad)
        touched = bad.view(-1, 32).any(1)
        assert torch.equal(getattr(h, s)[0][~touched], getattr(clean, s)[0][~touched])
        assert torch.equal(getattr(h, t)[0].view(-1, 32)[~touched], getattr(clean, t)[0].view(-1, 32)[~touched])
    assert torch.equal(h.params[0][~bad], clean.params[0][~bad]) and torch.isnan(h.params[0][bad]).all()


@pytest.mark.parametrize("mx", [False, True])
def test_adamw_skips_a_step_whose_scale_is_not_finite(mx):
    for bad in (float("inf"), float("nan")):
        p, gr = torch.ones(100, device="cuda"), torch.ones(100, device="cuda")
        h = moe.adamw_tensors([p], [gr], mxfp8=mx)
        moe.moe_adamw(h, 1, grad_scale=torch.tensor(bad, device="cuda").view(1), **HYPER)
        assert (p == 1).all() and not h.m[0].any() and not h.v[0].any()


def test_adamw_non_finite_gradients_show():
    for mx in (False, True):
        p, gr = torch.ones(96, device="cuda"), torch.full((96,), 0.5, device="cuda")
        gr[3], gr[40] = float("nan"), float("inf")
        h = moe.adamw_tensors([p], [gr], mxfp8=mx)
        moe.moe_adamw(h, 1, **HYPER)
        bad = torch.isnan(p)
        assert bad[3] and bad[40] and int(bad.sum()) == 2
        if mx:  # kept as NaN in the states; finite neighbours of the NaN are not disturbed
            m = mx_decode(h.m[0], h.m_scale[0])
            assert torch.isnan(m[3]) and torch.isnan(m[40]) and not torch.isnan(m[:3]).any()


# ------------------------------------------------------------------ streams, graphs
def test_training_calls_on_another_stream_and_in_a_graph():
    g, shape, ids, w = token_case(40, 64, 64, 0, 4, 0, 256)
    x, b, res = randn(g, 40, 256, dtype=BF), randn(g, 256), randn(g, 40, 256, dtype=BF)
    ws, ln_ws = moe.token_map_workspace(shape), moe.layer_norm_workspace(40, 256)

    def chain():
        y, h, mean, rstd = moe.moe_layer_norm(x, b, b, res)
        maps = moe.moe_token_map(shape, ids, ws=ws)
        rows = moe.moe_permute(shape, y, maps)
        out = moe.moe_unpermute(shape, rows, w, maps)
        dy, dw = moe.moe_unpermute_backward(shape, out, rows, w, maps)
        dx = moe.moe_permute_backward(shape, dy, maps)
        dl, _ = moe.moe_route_backward(shape, ids, w, dw)
        return (out, dw, dl) + moe.moe_layer_norm_backward(dx, h, mean, rstd, b, dh=out, ws=ln_ws)

    want = chain()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = chain()
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = chain()
    x.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(held, chain()))


def test_adamw_in_a_graph():
    p, gr = torch.ones(1000, device="cuda"), torch.ones(1000, device="cuda")
    h = moe.adamw_tensors([p], [gr])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_adamw(h, 5, **HYPER)
    graph.replay()
    torch.cuda.synchronize()
    assert math.isclose(h.m[0][0].item(), 0.1, rel_tol=1e-6) and p[0].item() < 1
