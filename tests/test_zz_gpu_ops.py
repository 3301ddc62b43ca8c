"""The layer operators on the GPU against plain 64-bit arithmetic: quantised rows, integer products with
scales (dense and by expert), MoE sort, dispatch, combine and its gradients.

Tolerances count roundings: half a step of the output type (finfo.eps / 2), 2^-24 for every fp32
operation. Integers, positions and moved rows are compared exactly. The file is named so that pytest
collects it after the proof suites.
"""

import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24  # half a step of fp32


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sum_check_prover_b200 import build
    build.build()
    import sum_check_prover_b200 as fp
    ctx = fp.Context(0)
    yield torch, fp, ctx
    ctx.close()


def half_step(torch, t):
    return torch.finfo(t).eps / 2


def within(got, want, rel, absolute=0.0):
    """|got - want| <= rel |want| + absolute, element by element, NaN and infinities in the same places."""
    got, want = got.double().cpu().numpy(), np.asarray(want, dtype=np.float64)
    assert got.shape == want.shape
    assert np.array_equal(np.isnan(got), np.isnan(want))
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
    err = np.abs(got - want)[fine]
    bound = (rel * np.abs(want) + absolute)[fine]
    assert (err <= bound).all(), (err - bound).max()


def wide(torch, rows, cols, pad, dtype, lead=0):
    """rows x cols as part of a wider buffer that starts `lead` elements into its allocation; the
    buffer is filled with a pattern and returned too, to see that nothing else is written."""
    buf = torch.full((max(1, rows) * (cols + pad) + lead,), 7, dtype=dtype, device="cuda")
    return buf[lead:lead + rows * (cols + pad)].view(rows, cols + pad)[:, :cols], buf


def untouched(torch, view, buf, before):
    """Nothing of buf but view's elements differs from `before`."""
    mask = torch.ones_like(buf, dtype=torch.bool)
    off = view.storage_offset()
    if view.numel():
        mask.as_strided(view.shape, view.stride(), off).fill_(False)
    assert torch.equal(buf[mask], before[mask])


# ---- quantised rows -------------------------------------------------------------------------

def quantized(x):
    """q and scale of float64 rows that hold the inputs' values, exactly rounded."""
    q = np.zeros(x.shape, dtype=np.int8)
    s = np.zeros(len(x), dtype=np.float32)
    for t, row in enumerate(x):
        if not np.isfinite(row).all():
            s[t] = np.nan
            continue
        a = np.abs(row).max() if row.size else 0.0
        s[t] = np.float32(a) / np.float32(127)
        if a > 0:
            q[t] = np.rint(row * 127 / a)
    return q, s


TYPES = ["float32", "float16", "bfloat16"]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K,pad,lead", [(1, 1, 0, 0), (1, 7, 0, 0), (3, 64, 0, 0), (5, 129, 0, 1), (2, 1024, 16, 0),
                                          (150, 257, 3, 0), (7, 5120, 0, 0), (2, 16384, 8, 0), (3, 40000, 0, 0),
                                          (2, 33001, 0, 1), (1100, 96, 0, 0), (40, 256, 3, 1), (3, 9008, 5, 2)])
def test_quantize_rows(env, dtype, T, K, pad, lead):
    torch, fp, ctx = env
    dt = getattr(torch, dtype)
    g = torch.Generator(device="cuda").manual_seed(T * 131 + K)
    x, _ = wide(torch, T, K, pad, dt, lead)
    x.copy_(torch.randn(T, K, generator=g, device="cuda") * torch.exp(torch.randn(T, 1, generator=g, device="cuda")))
    q, qb = wide(torch, T, K, pad, torch.int8, lead)
    before, scale = qb.clone(), torch.empty(T, device="cuda")
    ctx.quantize_rows(x, q, scale)
    wq, ws = quantized(x.double().cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), wq)
    assert np.array_equal(scale.cpu().numpy(), ws)
    untouched(torch, q, qb, before)


def test_quantize_ties_and_borders(env):
    # 127 x / a at n + 1/2 exactly (a = 127 * 2^s, x = (n + 1/2) 2^s), one step of fp32 to either side of
    # it, and a = odd numbers where 254 x = (2 n + 1) a has solutions
    torch, fp, ctx = env
    rows = []
    for s in (-140, -126, -80, -10, 0, 60, 100):
        n = np.arange(-127, 127)
        mid = np.ldexp((n + 0.5).astype(np.float64), s).astype(np.float32)
        up, down = np.nextafter(mid, np.float32(np.inf)), np.nextafter(mid, np.float32(-np.inf))
        rows.append(np.concatenate([[np.float32(np.ldexp(127.0, s))], mid, up, down]).astype(np.float32))
    width = len(rows[0])
    for a in (254.0, 254.0 * 3, 2.0 ** -149, 2.0 ** -148 * 127, 3.4e38, 1e-40):
        a = np.float32(a)
        r = (np.arange(width) / width * a).astype(np.float32)
        r[0], r[1] = a, -a
        rows.append(r)
    x = np.stack(rows)
    xt = torch.from_numpy(x).cuda()
    for view in (xt, wide(torch, *x.shape, 1, torch.float32)[0].copy_(xt)):  # the wide and the narrow loads
        q, s = torch.zeros(x.shape, dtype=torch.int8, device="cuda"), torch.empty(len(x), device="cuda")
        ctx.quantize_rows(view, q, s)
        wq, ws = quantized(x.astype(np.float64))
        assert np.array_equal(q.cpu().numpy(), wq)
        assert np.array_equal(s.cpu().numpy(), ws)


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_zero_and_unfinite_rows(env, dtype):
    torch, fp, ctx = env
    x = torch.randn(6, 48, device="cuda").to(getattr(torch, dtype))
    x[0] = 0
    x[1] = -0.0
    x[2, 5] = math.nan
    x[3, 47] = math.inf
    x[4, 0] = -math.inf
    q, s = torch.full((6, 48), 9, dtype=torch.int8, device="cuda"), torch.empty(6, device="cuda")
    ctx.quantize_rows(x, q, s)
    wq, ws = quantized(x.double().cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), wq)
    assert np.array_equal(s.cpu().numpy(), ws, equal_nan=True)


@pytest.mark.parametrize("T,K,k,R", [(5, 32, 1, 5), (9, 33, 3, 40), (70, 256, 2, 140)])
def test_quantize_to_rows(env, T, K, k, R):
    torch, fp, ctx = env
    rng = np.random.default_rng(T)
    x = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).cuda().bfloat16()
    pos = rng.permutation(R)[:T * k].reshape(T, k).astype(np.int32)
    pos[rng.random((T, k)) < 0.2] = -1
    pos[0, 0] = R  # outside: passed over
    if T > 1:
        pos[1, 0] = 2 ** 31 - 1
    q, s = torch.full((R, K), 3, dtype=torch.int8, device="cuda"), torch.full((R,), 5.0, device="cuda")
    ctx.quantize_rows(x, q, s, pos=torch.from_numpy(pos).cuda())
    xq, xs = quantized(x.double().cpu().numpy())
    wq, ws = np.full((R, K), 3, dtype=np.int8), np.full(R, 5.0, dtype=np.float32)
    for t in range(T):
        for p in pos[t]:
            if 0 <= p < R:
                wq[p], ws[p] = xq[t], xs[t]
    assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(s.cpu().numpy(), ws)


# ---- integer products -----------------------------------------------------------------------

def product_case(torch, N, M, K, E, dtype, seed, padw=0, padx=0, pady=0, lead=0, extreme=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if E:
        w = torch.randint(-128, 128, (E, M, K), generator=g, device="cuda", dtype=torch.int8)
    else:
        w, _ = wide(torch, M, K, padw, torch.int8, lead)
        w.copy_(torch.randint(-128, 128, (M, K), generator=g, device="cuda", dtype=torch.int8))
    x, _ = wide(torch, N, K, padx, torch.int8, lead)
    x.copy_(torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8))
    if extreme:
        w.fill_(-128)
        x.fill_(-128)
    ws = torch.exp(torch.randn((E, M) if E else (M,), generator=g, device="cuda")) * 1e-3
    xs = torch.exp(torch.randn(N, generator=g, device="cuda")) * 1e-2
    y, yb = wide(torch, N, M, pady, getattr(torch, dtype), lead)
    return w, x, ws, xs, y, yb


def check_product(torch, w, x, ws, xs, y, ends=None):
    """y against the exact sums (float64 holds them) times both scales."""
    wn, xn = w.double().cpu().numpy(), x.double().cpu().numpy()
    wsn, xsn = ws.double().cpu().numpy(), xs.double().cpu().numpy()
    # the sum to fp32, two products, and the rounding to y's type (f16 below its normal numbers: half
    # of its smallest step)
    rel = 4 * U + half_step(torch, y.dtype)
    tiny = torch.finfo(y.dtype).smallest_normal * torch.finfo(y.dtype).eps / 2
    if ends is None:
        within(y, (xn @ wn.T) * xsn[:, None] * wsn, rel, tiny)
        return
    for e, (a, b) in enumerate(zip(ends, ends[1:])):
        if a < b:
            within(y[a:b], (xn[a:b] @ wn[e].T) * xsn[a:b, None] * wsn[e], rel, tiny)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,M,K", [(1, 1, 1), (1, 128, 64), (1, 300, 5120), (2, 129, 17), (15, 64, 128), (16, 200, 256),
                                   (17, 1000, 96), (33, 130, 1000), (64, 256, 2048), (65, 257, 129), (128, 384, 640),
                                   (129, 127, 1024), (200, 640, 4096), (256, 128, 128), (257, 512, 272), (700, 300, 512)])
def test_matmul_dense(env, dtype, N, M, K):
    torch, fp, ctx = env
    w, x, ws, xs, y, yb = product_case(torch, N, M, K, 0, dtype, N + M + K)
    ctx.matmul_i8(w, x, y, ws, xs)
    check_product(torch, w, x, ws, xs, y)


@pytest.mark.parametrize("padw,padx,pady,lead", [(16, 0, 0, 0), (0, 16, 5, 0), (3, 0, 0, 0), (0, 3, 0, 0), (5, 1, 3, 0),
                                                 (0, 0, 0, 1), (16, 16, 8, 16), (4, 4, 0, 4), (13, 8, 1, 2)])
@pytest.mark.parametrize("N,M,K", [(1, 70, 80), (40, 200, 333), (300, 150, 400)])
def test_matmul_strides(env, N, M, K, padw, padx, pady, lead):
    torch, fp, ctx = env
    w, x, ws, xs, y, yb = product_case(torch, N, M, K, 0, "bfloat16", 5, padw, padx, pady, lead)
    before = yb.clone()
    ctx.matmul_i8(w, x, y, ws, xs)
    check_product(torch, w, x, ws, xs, y)
    untouched(torch, y, yb, before)


def test_matmul_largest_sums(env):
    # K = 131071 of (-128)^2: the sum 2^14 K is the largest the int32 holds
    torch, fp, ctx = env
    w, x, ws, xs, y, yb = product_case(torch, 3, 5, 131071, 0, "float32", 1, extreme=True)
    ctx.matmul_i8(w, x, y, ws, xs)
    check_product(torch, w, x, ws, xs, y)


@pytest.mark.parametrize("K", [5120, 4100])
@pytest.mark.parametrize("N", [1, 8, 40, 100])
def test_matmul_few_rows_of_weights(env, N, K):
    # few output tiles: the sums over K are split among blocks
    torch, fp, ctx = env
    for M in (64, 129, 640):
        w, x, ws, xs, y, yb = product_case(torch, N, M, K, 0, "float16", N + M)
        ctx.matmul_i8(w, x, y, ws, xs)
        check_product(torch, w, x, ws, xs, y)


@pytest.mark.parametrize("counts", [[1], [0, 3, 0, 1], [5, 0, 0, 0], [0, 0, 0, 7], [16, 17, 31, 33, 1], [130, 2, 257, 0, 40],
                                    [300] * 3, [0] * 40 + [2] + [0] * 23, [1] * 64])
@pytest.mark.parametrize("M,K", [(64, 64), (200, 272), (130, 333)])
def test_matmul_by_expert(env, counts, M, K):
    torch, fp, ctx = env
    E, N = len(counts), sum(counts) + 3  # three rows that no expert has
    w, x, ws, xs, y, yb = product_case(torch, N, M, K, E, "bfloat16", E + M)
    ends = np.concatenate([[0], np.cumsum(counts)])
    y.fill_(7)
    ctx.matmul_i8(w, x, y, ws, xs, offsets=torch.from_numpy(ends.astype(np.int32)).cuda())
    check_product(torch, w, x, ws, xs, y, ends)
    assert bool((y[ends[-1]:] == 7).all())


def test_matmul_offsets_are_kept_inside(env):
    # rows before the first offset and past the last are left; offsets outside [0, N] or falling are clamped
    torch, fp, ctx = env
    w, x, ws, xs, y, yb = product_case(torch, 20, 40, 64, 4, "float32", 3)
    for off, ends in (([4, 9, 9, 12, 15], [4, 9, 9, 12, 15]), ([-5, 3, 2, 30, 2 ** 31 - 1], [0, 3, 3, 20, 20])):
        y.fill_(7)
        ctx.matmul_i8(w, x, y, ws, xs, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
        if off[0] >= 0:
            check_product(torch, w, x, ws, xs, y, ends)
            assert bool((y[:4] == 7).all()) and bool((y[15:] == 7).all())
        else:
            check_product(torch, w[:1], x[:3], ws[:1], xs[:3], y[:3], [0, 3])
    y.fill_(7)
    ctx.matmul_i8(w, x, y, ws, xs, offsets=torch.zeros(5, dtype=torch.int32, device="cuda"))
    assert bool((y == 7).all())
    ctx.matmul_i8(w, x[:0], y[:0], ws, xs[:0], offsets=torch.zeros(5, dtype=torch.int32, device="cuda"))


def test_matmul_one_group_with_offsets(env):
    # one expert, with offsets that leave rows out at both ends
    torch, fp, ctx = env
    w, x, ws, xs, y, yb = product_case(torch, 50, 100, 96, 1, "float32", 4)
    y.fill_(7)
    ctx.matmul_i8(w, x, y, ws, xs, offsets=torch.tensor([7, 45], dtype=torch.int32, device="cuda"))
    check_product(torch, w, x, ws, xs, y, [7, 45])
    assert bool((y[:7] == 7).all()) and bool((y[45:] == 7).all())


def test_matmul_many_experts(env):
    torch, fp, ctx = env
    rng = np.random.default_rng(0)
    E, M, K = 4096, 16, 32
    counts = (rng.random(E) < 0.05) * rng.integers(1, 20, E)
    N = int(counts.sum())
    w, x, ws, xs, y, yb = product_case(torch, N, M, K, E, "float32", 9)
    ends = np.concatenate([[0], np.cumsum(counts)])
    ctx.matmul_i8(w, x, y, ws, xs, offsets=torch.from_numpy(ends.astype(np.int32)).cuda())
    check_product(torch, w, x, ws, xs, y, ends)


def test_matmul_nan_scales_stay_in_their_rows(env):
    torch, fp, ctx = env
    w, x, ws, xs, y, yb = product_case(torch, 40, 150, 128, 0, "bfloat16", 11)
    xs[3], xs[39], ws[149] = math.nan, math.inf, math.nan
    x[3] = 0
    ctx.matmul_i8(w, x, y, ws, xs)
    got = y.float().cpu().numpy()
    assert np.isnan(got[3]).all() and np.isnan(got[:, 149]).all()
    ok = np.ones(40, bool)
    ok[[3, 39]] = False
    check_product(torch, w[:149], x[torch.from_numpy(ok).cuda()], ws[:149], xs[torch.from_numpy(ok).cuda()],
                  y[torch.from_numpy(ok).cuda()][:, :149])


def test_matmul_pitches_past_32_bits(env):
    torch, fp, ctx = env
    K, M, ld = 128, 40, (1 << 31) + 48
    xb = torch.empty(ld + K, dtype=torch.int8, device="cuda")
    yb = torch.empty(ld + M, dtype=torch.bfloat16, device="cuda")
    x, y = xb.as_strided((2, K), (ld, 1)), yb.as_strided((2, M), (ld, 1))
    x.copy_(torch.randint(-128, 128, (2, K), device="cuda"))
    w = torch.randint(-128, 128, (M, K), device="cuda", dtype=torch.int8)
    wl = xb.new_empty(ld + K).as_strided((2, K), (ld, 1))
    wl.copy_(w[:2])
    ws, xs = torch.rand(M, device="cuda"), torch.rand(2, device="cuda")
    ctx.matmul_i8(w, x, y, ws, xs)
    check_product(torch, w, x, ws, xs, y)
    ctx.matmul_i8(wl, x, y[:, :2], ws[:2], xs)
    check_product(torch, wl, x, ws[:2], xs, y[:, :2])


# ---- sort -----------------------------------------------------------------------------------

def sorted_choices(e, E):
    key = np.where((e.reshape(-1) >= 0) & (e.reshape(-1) < E), e.reshape(-1), E)
    order = np.argsort(key, kind="stable")
    pos = np.empty(len(key), dtype=np.int32)
    pos[order] = np.arange(len(key))
    pos[key == E] = -1
    return np.array([(key < x).sum() for x in range(E)] + [(key < E).sum()], dtype=np.int32), pos.reshape(e.shape)


@pytest.mark.parametrize("n,E", [(0, 5), (1, 1), (1, 4096), (31, 3), (32, 128), (33, 128), (1000, 7), (1025, 128), (4097, 4096),
                                 (8192, 128), (16384, 1), (16384, 256), (100003, 60), (300000, 4096)])
@pytest.mark.parametrize("kind", ["even", "skewed", "one", "none"])
def test_moe_sort(env, n, E, kind):
    torch, fp, ctx = env
    rng = np.random.default_rng(n + E)
    e = {"even": lambda: rng.integers(0, E, n), "skewed": lambda: np.minimum(E - 1, rng.geometric(0.2, n) - 2),
         "one": lambda: np.full(n, E - 1), "none": lambda: np.where(rng.random(n) < 0.5, -1, E + 3)}[kind]().astype(np.int32)
    if kind == "even" and n > 3:
        e[1], e[2] = -2 ** 31, 2 ** 31 - 1
    off = torch.full((E + 1,), -9, dtype=torch.int32, device="cuda")
    pos = torch.full((n,), -9, dtype=torch.int32, device="cuda")
    ctx.moe_sort(torch.from_numpy(e).cuda(), E, off, pos)
    wo, wp = sorted_choices(e, E)
    assert np.array_equal(off.cpu().numpy(), wo)
    assert np.array_equal(pos.cpu().numpy(), wp)


# ---- dispatch and combine -------------------------------------------------------------------

def routed(rng, T, k, E, R=None, drop=0.1):
    """Positions as the sort gives them, some choices dropped."""
    e = rng.integers(0, E, (T, k)).astype(np.int32)
    e[rng.random((T, k)) < drop] = -1
    return sorted_choices(e, E)[1]


@pytest.mark.parametrize("dtype,K,pad,lead", [("int8", 1, 0, 0), ("int8", 33, 0, 0), ("int8", 64, 0, 0), ("int8", 40, 0, 1), ("bfloat16", 8, 0, 0),
                                              ("bfloat16", 513, 1, 0), ("float32", 100, 0, 0), ("float32", 5, 3, 1), ("float16", 2048, 8, 0), ("bfloat16", 64, 3, 1), ("int8", 160, 5, 7), ("float32", 40, 3, 1),
                                              ("int64", 3, 0, 0)])
@pytest.mark.parametrize("T,k", [(1, 8), (40, 1), (300, 3)])
def test_moe_dispatch(env, dtype, K, pad, lead, T, k):
    torch, fp, ctx = env
    dt = getattr(torch, dtype)
    rng = np.random.default_rng(T + K)
    pos = routed(rng, T, k, 8)
    x, _ = wide(torch, T, K, pad, dt, lead)
    x.copy_(torch.from_numpy(rng.integers(-100, 100, (T, K))).cuda())
    rows, rb = wide(torch, T * k, K, pad, dt, lead)
    before = rb.clone()
    want = rows.cpu().numpy().copy() if dtype != "bfloat16" else rows.float().cpu().numpy().copy()
    xs = x.cpu().numpy() if dtype != "bfloat16" else x.float().cpu().numpy()
    for t in range(T):
        for p in pos[t]:
            if p >= 0:
                want[p] = xs[t]
    ctx.moe_dispatch(x, torch.from_numpy(pos).cuda(), rows)
    got = rows.cpu().numpy() if dtype != "bfloat16" else rows.float().cpu().numpy()
    assert np.array_equal(got, want)
    untouched(torch, rows, rb, before)


def combined(rows, pos, w, base):
    """The sums in 64 bits, and the sums of magnitudes that bound their rounding."""
    T, k = pos.shape
    out = np.zeros((T, rows.shape[1])) if base is None else base.copy()
    mag = np.abs(out)
    for t in range(T):
        for j in range(k):
            if 0 <= pos[t, j] < len(rows):
                v = rows[pos[t, j]] * (1.0 if w is None else float(w[t, j]))
                out[t] += v
                mag[t] += np.abs(v)
    return out, mag


@pytest.mark.parametrize("rt,ot", [(a, b) for a in TYPES for b in TYPES])
@pytest.mark.parametrize("T,k,M,pad,lead", [(1, 8, 64, 0, 0), (3, 1, 1, 0, 0), (37, 2, 333, 0, 0), (64, 3, 256, 8, 0), (20, 9, 130, 3, 1), (33, 2, 256, 3, 0)])
@pytest.mark.parametrize("weighted,based", [(True, True), (False, False)])
def test_moe_combine(env, rt, ot, T, k, M, pad, lead, weighted, based):
    torch, fp, ctx = env
    rng = np.random.default_rng(T + M)
    pos = routed(rng, T, k, 4)
    R = T * k
    rows, _ = wide(torch, R, M, pad, getattr(torch, rt), lead)
    rows.copy_(torch.from_numpy(rng.standard_normal((R, M))).cuda())
    rows[int((pos >= 0).sum()):] = math.nan  # behind the last row: never read
    w = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda() if weighted else None
    out, ob = wide(torch, T, M, pad, getattr(torch, ot), lead)
    base = None
    if based:
        base, _ = wide(torch, T, M, pad, getattr(torch, ot), lead)
        base.copy_(torch.from_numpy(rng.standard_normal((T, M))).cuda())
    before = ob.clone()
    ctx.moe_combine(rows, torch.from_numpy(pos).cuda(), out, weights=w, base=base)
    want, mag = combined(rows.double().cpu().numpy(), pos, None if w is None else w.cpu().numpy(),
                         None if base is None else base.double().cpu().numpy())
    # k + 1 fp32 additions at most, each of a sum no larger than the magnitudes', then y's rounding
    err, h = (k + 2) * U * mag, half_step(torch, out.dtype)
    tiny = torch.finfo(out.dtype).smallest_normal * torch.finfo(out.dtype).eps / 2
    within(out, want, h, err * (1 + h) + tiny)
    untouched(torch, out, ob, before)
    if based:  # onto the base itself
        ctx.moe_combine(rows, torch.from_numpy(pos).cuda(), base, weights=w, base=base)
        assert torch.equal(base, out)


def test_moe_combine_tokens_without_rows(env):
    torch, fp, ctx = env
    rows = torch.full((4, 40), math.nan, device="cuda")
    pos = torch.tensor([[-1, -1], [4, 2 ** 31 - 1], [-2 ** 31, -1]], dtype=torch.int32, device="cuda")
    out = torch.full((3, 40), 5.0, device="cuda")
    ctx.moe_combine(rows, pos, out, weights=torch.full((3, 2), math.nan, device="cuda"))
    assert bool((out == 0).all())
    dw, dr = torch.full((3, 2), 9.0, device="cuda"), torch.full((4, 40), 3.0, device="cuda")
    ctx.moe_combine_grad(torch.full((3, 40), math.nan, device="cuda"), rows, pos, None, dr, dw)
    assert bool((dw == 0).all()) and bool((dr == 3).all())
    ctx.moe_combine(rows[:0], pos, out)  # no rows at all
    assert bool((out == 0).all())
    empty = pos[:0]
    ctx.moe_combine(rows, empty, out[:0])
    ctx.moe_combine_grad(out[:0], rows, empty, None, dr, dw[:0])
    ctx.moe_dispatch(out[:0], empty, rows)
    assert bool(rows.isnan().all())


@pytest.mark.parametrize("rt,ot", [("float32", "float32"), ("bfloat16", "bfloat16"), ("float16", "float32"), ("float32", "bfloat16"),
                                   ("bfloat16", "float16")])
@pytest.mark.parametrize("T,k,M,pad,lead", [(1, 8, 64, 0, 0), (2, 1, 1, 0, 0), (37, 2, 333, 0, 0), (50, 5, 2048, 8, 0), (9, 3, 130, 3, 1), (33, 4, 256, 3, 0), (1, 7, 1000, 3, 0)])
def test_moe_combine_grad(env, rt, ot, T, k, M, pad, lead):
    torch, fp, ctx = env
    rng = np.random.default_rng(T + M)
    pos = routed(rng, T, k, 4)
    R = T * k + 2
    rows, _ = wide(torch, R, M, pad, getattr(torch, rt), lead)
    rows.copy_(torch.from_numpy(rng.standard_normal((R, M))).cuda())
    dout, _ = wide(torch, T, M, pad, getattr(torch, ot), lead)
    dout.copy_(torch.from_numpy(rng.standard_normal((T, M))).cuda())
    w = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    drows, rb = wide(torch, R, M, pad, getattr(torch, rt), lead)
    before, dw = rb.clone(), torch.full((T, k), 9.0, device="cuda")
    p = torch.from_numpy(pos).cuda()
    ctx.moe_combine_grad(dout, rows, p, w, drows, dw)
    g, r, wn = dout.double().cpu().numpy(), rows.double().cpu().numpy(), w.double().cpu().numpy()
    want, wdw, mag = np.full((R, M), 7.0), np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            if pos[t, j] >= 0:
                want[pos[t, j]] = wn[t, j] * g[t]
                wdw[t, j] = g[t] @ r[pos[t, j]]
                mag[t, j] = np.abs(g[t]) @ np.abs(r[pos[t, j]])
    h = half_step(torch, rows.dtype)
    tiny = torch.finfo(rows.dtype).smallest_normal * torch.finfo(rows.dtype).eps / 2
    within(drows, want, (1 + U) * (1 + h) - 1, tiny)
    # at least 32 partial sums: M / 32 additions in one, and the joining of at most 1024 and the last
    within(dw, wdw, 0.0, (math.ceil(M / 32) + 8 + 16) * U * mag)
    untouched(torch, drows, rb, before)
    d2, dw2 = drows.clone(), torch.empty_like(dw)
    ctx.moe_combine_grad(dout, rows, p, w, dweights=dw2)
    ctx.moe_combine_grad(dout, rows, p, w, drows=d2)
    assert torch.equal(dw2, dw) and torch.equal(d2, drows)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,lead", [(3, 0), (1, 1), (5, 2), (7, 3)])
def test_odd_inputs_dense_outputs(env, dtype, pad, lead):
    # every input in rows of odd pitches, the outputs dense: loads from any address, to the matrices' ends
    torch, fp, ctx = env
    dt = getattr(torch, dtype)
    rng = np.random.default_rng(pad)
    T, k, M = 21, 2, 304

    def odd(n):
        t, _ = wide(torch, n, M, pad, dt, lead)
        return t.copy_(torch.from_numpy(rng.standard_normal((n, M))).cuda())

    x, rows, dout, base = odd(T), odd(T * k), odd(T), odd(T)
    pos = torch.from_numpy(routed(rng, T, k, 4)).cuda()
    w = torch.from_numpy(rng.random((T, k)).astype(np.float32)).cuda()

    def run(x, rows, dout, base):
        q, s = torch.zeros(T * k, M, dtype=torch.int8, device="cuda"), torch.zeros(T * k, device="cuda")
        ctx.quantize_rows(x, q, s, pos=pos)
        d, out = torch.zeros(T * k, M, dtype=dt, device="cuda"), torch.zeros(T, M, dtype=dt, device="cuda")
        ctx.moe_dispatch(x, pos, d)
        ctx.moe_combine(rows, pos, out, weights=w, base=base)
        dr, dw = torch.zeros(T * k, M, dtype=dt, device="cuda"), torch.zeros(T, k, device="cuda")
        ctx.moe_combine_grad(dout, rows, pos, w, dr, dw)
        return q, s, d, out, dr, dw

    for got, want in zip(run(x, rows, dout, base), run(*(t.contiguous() for t in (x, rows, dout, base)))):
        assert torch.equal(got, want)


def test_gradients_against_differences(env):
    # small integers, so that every fp32 sum is exact: the layer is linear in the rows, the weights and the
    # tokens, and each gradient is the difference that one step in its direction makes
    torch, fp, ctx = env
    rng = np.random.default_rng(2)
    T, k, M = 6, 3, 40
    pos = torch.from_numpy(routed(rng, T, k, 3, drop=0.3)).cuda()
    R = T * k

    def ints(*s):
        return torch.from_numpy(rng.integers(-4, 5, s).astype(np.float32)).cuda()

    x, w, dout = ints(T, M), ints(T, k), ints(T, M)

    def loss(x, w, rows=None):
        if rows is None:
            rows = torch.zeros(R, M, device="cuda")
            ctx.moe_dispatch(x, pos, rows)
        out = torch.empty(T, M, device="cuda")
        ctx.moe_combine(rows, pos, out, weights=w)
        return float((out.double() * dout.double()).sum())

    rows = torch.zeros(R, M, device="cuda")
    ctx.moe_dispatch(x, pos, rows)
    drows, dw, dx = torch.zeros(R, M, device="cuda"), torch.empty(T, k, device="cuda"), torch.empty(T, M, device="cuda")
    ctx.moe_combine_grad(dout, rows, pos, w, drows, dw)
    ctx.moe_combine(drows, pos, dx)  # the dispatch's gradient: a token's rows summed
    at = loss(x, w)
    for t in range(T):
        for j in range(k):
            w2 = w.clone()
            w2[t, j] += 1
            assert loss(x, w2) - at == float(dw[t, j])
        for m in (0, 17, M - 1):
            x2 = x.clone()
            x2[t, m] += 1
            assert loss(x2, w) - at == float(dx[t, m])
    for r in range(R):
        r2 = rows.clone()
        r2[r, 5] += 1
        assert loss(x, w, r2) - at == float(drows[r, 5])


# ---- together -------------------------------------------------------------------------------

def layer(torch, ctx, s, stream=None):
    """An 8-bit MoE layer: tokens quantised into their experts' rows, gate and up products, the gated
    product (torch), quantised again, the down product, and back with the router's weights."""
    ctx.moe_sort(s["e"], s["E"], s["offsets"], s["pos"], stream=stream)
    ctx.quantize_rows(s["x"], s["xq"], s["xs"], pos=s["pos"], stream=stream)
    ctx.matmul_i8(s["w1"], s["xq"], s["h"], s["w1s"], s["xs"], offsets=s["offsets"], stream=stream)
    F = s["w2"].shape[2]
    torch.mul(torch.nn.functional.silu(s["h"][:, :F]), s["h"][:, F:], out=s["a"])
    ctx.quantize_rows(s["a"], s["aq"], s["as"], stream=stream)
    ctx.matmul_i8(s["w2"], s["aq"], s["z"], s["w2s"], s["as"], offsets=s["offsets"], stream=stream)
    ctx.moe_combine(s["z"], s["pos"], s["out"], weights=s["weights"], base=s["shared"], stream=stream)
    return s["out"]


def layer_state(torch, T, k, E, d, F, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    R = T * k

    def i8(*s):
        return torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int8)

    def z(*s, dtype=torch.float32):
        return torch.zeros(*s, dtype=dtype, device="cuda")

    e = torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32)
    e[0] = -1  # a token of padding
    return dict(E=E, e=e.contiguous(), x=torch.randn(T, d, generator=g, device="cuda").bfloat16(), w1=i8(E, 2 * F, d), w2=i8(E, d, F),
                w1s=torch.rand(E, 2 * F, generator=g, device="cuda") * 1e-3, w2s=torch.rand(E, d, generator=g, device="cuda") * 1e-3,
                weights=torch.rand(T, k, generator=g, device="cuda"), shared=torch.randn(T, d, generator=g, device="cuda").bfloat16(),
                offsets=z(E + 1, dtype=torch.int32), pos=z(T, k, dtype=torch.int32), xq=z(R, d, dtype=torch.int8), xs=z(R), h=z(R, 2 * F),
                a=z(R, F), aq=z(R, F, dtype=torch.int8), z=z(R, d), out=z(T, d, dtype=torch.bfloat16), **{"as": z(R)})


def layer_64(torch, s):
    """The same layer in 64 bits from its definition, token by token; the quantised values from the
    kernel's own activations (s["a"]), so that a rounding's border does not count."""
    x, out = s["x"].double().cpu().numpy(), s["shared"].double().cpu().numpy()
    e, F = s["e"].cpu().numpy(), s["w2"].shape[2]
    pos, h, a = s["pos"].cpu().numpy(), s["h"].double().cpu().numpy(), s["a"].double().cpu().numpy()
    mag = np.abs(out)
    for t in range(len(x)):
        q, sc = quantized(x[t:t + 1])
        for j in range(e.shape[1]):
            if e[t, j] < 0:
                continue
            r, ex = pos[t, j], e[t, j]
            w1, w2 = s["w1"][ex].double().cpu().numpy(), s["w2"][ex].double().cpu().numpy()
            want = (w1 @ q[0]) * float(sc[0]) * s["w1s"][ex].double().cpu().numpy()
            assert (np.abs(h[r] - want) <= 4 * U * np.abs(want)).all()
            aq, asc = quantized(a[r:r + 1])
            z = (w2 @ aq[0]) * float(asc[0]) * s["w2s"][ex].double().cpu().numpy()
            out[t] += float(s["weights"][t, j]) * z
            mag[t] += np.abs(float(s["weights"][t, j]) * z)
    return out, mag


@pytest.mark.parametrize("T,k,E,d,F", [(1, 2, 4, 64, 96), (40, 2, 8, 128, 256), (100, 1, 4, 128, 256)])
def test_layer(env, T, k, E, d, F):
    torch, fp, ctx = env
    s = layer_state(torch, T, k, E, d, F, T)
    out = layer(torch, ctx, s)
    want, mag = layer_64(torch, s)
    h = half_step(torch, torch.bfloat16)
    within(out, want, h, (k + 6) * U * mag * (1 + h))


def test_experts_inputs_prove(env):
    # the rows that the sort and the dispatch make are the dispatch statement's
    import oracle
    torch, fp, ctx = env
    rng = np.random.default_rng(5)
    T, d, E = 200, 96, 6
    x = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).cuda()
    e = torch.from_numpy(rng.integers(0, E, T).astype(np.int32)).cuda()
    xq, xs = torch.empty(T, d, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    off, pos, D = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty_like(e), torch.empty_like(xq)
    ctx.quantize_rows(x, xq, xs)
    ctx.moe_sort(e, E, off, pos)
    ctx.moe_dispatch(xq, pos[:, None], D)
    D2, s2 = torch.empty_like(D), torch.empty_like(xs)
    ctx.quantize_rows(x, D2, s2, pos=pos[:, None])
    assert torch.equal(D, D2)
    tx = fp.Transcript(8)
    pf = ctx.prove_dispatch(tx, xq, e, D, E)
    args = (8, xq.cpu().numpy(), e.cpu().numpy(), D.cpu().numpy(), E)
    assert (pf, tx.state()) == oracle.dsp_prove(*args)
    assert oracle.dsp_verify(*args, pf)[0] == "accept"


def test_quantized_activations_prove(env):
    # a site over quantised activations: the proven integers are those of the scaled product
    torch, fp, ctx = env
    rng = np.random.default_rng(6)
    N, M, K, k = 24, 48, 128, 12
    x = torch.from_numpy(rng.standard_normal((N, K)).astype(np.float32)).cuda()
    w = torch.from_numpy(rng.integers(-128, 128, (M, K)).astype(np.int8)).cuda()
    xq, xs, y = torch.empty(N, K, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda"), torch.empty(N, M, device="cuda")
    ctx.quantize_rows(x, xq, xs)
    one = torch.ones(N, device="cuda")
    ctx.matmul_i8(w, xq, y, torch.ones(M, device="cuda"), one)
    q, r, y8 = (torch.empty(N, M, dtype=t, device="cuda") for t in (torch.int32, torch.int32, torch.int8))
    tx = fp.Transcript(1)
    ctx.commit_witness(tx, [fp.SiteDesc(w, xq, q, r, y8, M, K, N, 8, k)])
    assert torch.equal((q.long() << k) + r, y.long())  # |sums| < 2^24: exact in fp32


def test_graphs_and_streams(env):
    # two captured layers replayed side by side on streams of their own, on new inputs, give what plain
    # calls give
    torch, fp, ctx = env
    states = [layer_state(torch, 50, 2, 8, 128, 192, 20 + i) for i in range(2)]
    side = [torch.cuda.Stream() for _ in range(2)]
    graphs = []
    for s, st in zip(states, side):
        with torch.cuda.stream(st):
            layer(torch, ctx, s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            layer(torch, ctx, s)
        graphs.append(g)
    for trial in range(3):
        fresh = [layer_state(torch, 50, 2, 8, 128, 192, 100 + 10 * trial + i) for i in range(2)]
        want = [layer(torch, ctx, f).clone() for f in fresh]
        for s, f in zip(states, fresh):
            for name, t in f.items():
                if name != "E" and name not in ("out", "z", "h"):
                    s[name].copy_(t)
        torch.cuda.synchronize()
        for _ in range(3):
            for g, st in zip(graphs, side):
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        for s, w in zip(states, want):
            assert torch.equal(s["out"], w)


def test_capture_as_a_first_call(env):
    # a context and shapes that nothing has run before the capture, with timing switched on
    torch, fp, _ = env
    ctx = fp.Context(0)
    try:
        s = layer_state(torch, 30, 2, 4, 96, 80, 3)
        ctx.set_profiling(2)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer(torch, ctx, s)
        g.replay()
        torch.cuda.synchronize()
        got = s["out"].clone()
        assert ctx.kernel_stats() == {}
        s["out"].zero_()
        assert torch.equal(layer(torch, ctx, s), got)
        stats = ctx.kernel_stats()
        assert {"quant_rows", "matmul_i8", "moe_sort", "moe_combine"} <= set(stats)
        ctx.set_profiling(0)
    finally:
        ctx.close()


def test_odd_pitches_in_graphs(env):
    # products whose operands are realigned in the stream's memory: plain, captured twice, replayed side by side
    torch, fp, ctx = env
    runs = []
    for i in range(2):
        w, x, ws, xs, y, yb = product_case(torch, 90 + i, 150, 333, 0, "float32", 40 + i, padx=3)
        st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=st):
            ctx.matmul_i8(w, x, y, ws, xs)
        runs.append((w, x, ws, xs, y, st, g))
    for _ in range(3):
        for w, x, ws, xs, y, st, g in runs:
            y.zero_()
            x.copy_(torch.randint(-128, 128, x.shape, device="cuda"))
        torch.cuda.synchronize()
        for _ in range(4):
            for w, x, ws, xs, y, st, g in runs:
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        for w, x, ws, xs, y, st, g in runs:
            check_product(torch, w, x, ws, xs, y)
            want = y.clone()
            ctx.matmul_i8(w, x, y, ws, xs)
            assert torch.equal(y, want)


@pytest.mark.parametrize("K", [65, 130, 268, 1032, 2047])  # pitches of 1, 2, 4, 8 and 15 modulo 16
@pytest.mark.parametrize("M", [64, 100, 1031, 2500])
@pytest.mark.parametrize("counts", [None, [1, 0, 3, 40], [0, 2, 0, 0, 1], [5]])
def test_weights_with_odd_pitches_and_few_tokens(env, K, M, counts):
    # weights read by classes of rows that begin at the same byte of 16, tokens shifted for each
    torch, fp, ctx = env
    E = 0 if counts is None else len(counts)
    N = 2 if counts is None else sum(counts) + 1
    w, x, ws, xs, y, yb = product_case(torch, N, M, K, E, "float32", K + M, pady=1)
    y.fill_(7)
    before = yb.clone()
    if E == 0:
        ctx.matmul_i8(w, x, y, ws, xs)
        check_product(torch, w, x, ws, xs, y)
    else:
        ends = np.concatenate([[0], np.cumsum(counts)])
        ctx.matmul_i8(w, x, y, ws, xs, offsets=torch.from_numpy(ends.astype(np.int32)).cuda())
        check_product(torch, w, x, ws, xs, y, ends)
        assert bool((y[ends[-1]:] == 7).all())
    untouched(torch, y, yb, before)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("padw,lead", [(3, 0), (8, 0), (1, 5), (0, 3)])
def test_weight_views_with_odd_pitches(env, dtype, padw, lead):
    torch, fp, ctx = env
    w, x, ws, xs, y, yb = product_case(torch, 7, 900, 640 if padw else 643, 0, dtype, 60, padw=padw, lead=lead)
    ctx.matmul_i8(w, x, y, ws, xs)
    check_product(torch, w, x, ws, xs, y)


def test_odd_pitches_by_expert(env):
    # experts without rows are not realigned; falling offsets do not hide one that has rows
    torch, fp, ctx = env
    for off, ends in (([0, 0, 5, 5, 9, 9], [0, 0, 5, 5, 9, 9]), ([0, 6, 2, 8, 8, 12], [0, 6, 6, 8, 8, 12])):
        w, x, ws, xs, y, yb = product_case(torch, 12, 50, 77, 5, "float32", 50)
        y.fill_(7)
        ctx.matmul_i8(w, x, y, ws, xs, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
        check_product(torch, w, x, ws, xs, y, ends)
        assert bool((y[ends[-1]:] == 7).all())


def test_other_stream_explicitly(env):
    torch, fp, ctx = env
    s = layer_state(torch, 64, 2, 8, 256, 256, 7)
    want = layer(torch, ctx, s).clone()
    s["z"].zero_()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    ctx.moe_sort(s["e"], s["E"], s["offsets"], s["pos"], stream=st)
    ctx.matmul_i8(s["w2"], s["aq"], s["z"], s["w2s"], s["as"], offsets=s["offsets"], stream=st)
    ctx.moe_combine(s["z"], s["pos"], s["out"], weights=s["weights"], base=s["shared"], stream=st.cuda_stream)
    st.synchronize()
    assert torch.equal(s["out"], want)


def test_two_streams_at_once(env):
    # plain calls of one context on two streams, products of every shape among them, give what they give alone
    torch, fp, ctx = env
    shapes = [(1, 640, 5120, 0), (40, 300, 1024, 0), (400, 520, 512, 0), (1500, 2100, 256, 0), (3, 900, 333, 3), (90, 200, 77, 1)]
    side = [torch.cuda.Stream() for _ in range(2)]
    work = []
    for i, (N, M, K, pad) in enumerate(shapes * 2):
        w, x, ws, xs, y, yb = product_case(torch, N, M, K, 0, "bfloat16", i, padx=pad)
        q, s = torch.empty(N, K, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
        work.append((w, x, ws, xs, y, x.float(), q, s, side[i % 2]))
    torch.cuda.synchronize()
    for _ in range(4):
        for w, x, ws, xs, y, xf, q, s, st in work:
            ctx.quantize_rows(xf, q, s, stream=st)
            ctx.matmul_i8(w, x, y, ws, xs, stream=st)
    torch.cuda.synchronize()
    for w, x, ws, xs, y, xf, q, s, st in work:
        check_product(torch, w, x, ws, xs, y)
        assert np.array_equal(q.cpu().numpy(), quantized(xf.double().cpu().numpy())[0])


def test_the_same_row_twice(env):
    # positions are the caller's: a row that two choices share is added twice and gets each one's gradient term
    torch, fp, ctx = env
    rows = torch.randn(3, 96, device="cuda")
    pos = torch.tensor([[1, 1], [2, 0]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 0.25], [1.0, 2.0]], device="cuda")
    out, dw = torch.empty(2, 96, device="cuda"), torch.empty(2, 2, device="cuda")
    ctx.moe_combine(rows, pos, out, weights=w)
    r = rows.double().cpu().numpy()
    within(out[0], 0.75 * r[1], 0.0, 4 * U * np.abs(r[1]))
    ctx.moe_combine_grad(out, rows, pos, w, dweights=dw)
    assert float(dw[0, 0]) == float(dw[0, 1])


def test_choices_beyond_a_few(env):
    # more choices a token than are kept at a time, and a token that chooses one expert often
    torch, fp, ctx = env
    rng = np.random.default_rng(8)
    T, k, E, M = 5, 70, 6, 48
    e = rng.integers(-1, E, (T, k)).astype(np.int32)
    e[2] = 4
    off, pos = sorted_choices(e, E)
    o, p = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda")
    ctx.moe_sort(torch.from_numpy(e).cuda(), E, o, p)
    assert np.array_equal(o.cpu().numpy(), off) and np.array_equal(p.cpu().numpy(), pos)
    x = torch.from_numpy(rng.integers(-8, 9, (T, M)).astype(np.float32)).cuda()
    rows, back = torch.zeros(T * k, M, device="cuda"), torch.empty(T, M, device="cuda")
    ctx.moe_dispatch(x, p, rows)
    ctx.moe_combine(rows, p, back)
    assert torch.equal(back, x * torch.from_numpy((e >= 0).sum(1)).cuda()[:, None])
    w = torch.from_numpy(rng.integers(-3, 4, (T, k)).astype(np.float32)).cuda()
    dr, dw = torch.zeros_like(rows), torch.empty(T, k, device="cuda")
    ctx.moe_combine_grad(x, rows, p, w, dr, dw)
    live = torch.from_numpy(e >= 0).cuda()
    assert torch.equal(dw, torch.where(live, (x * x).sum(1, keepdim=True), 0.0))
    want = torch.zeros_like(rows)
    want[p[live].long()] = (w[:, :, None] * x[:, None])[live]
    assert torch.equal(dr, want)


def test_repeats_give_the_same_bits(env):
    torch, fp, ctx = env
    s = layer_state(torch, 90, 3, 8, 160, 224, 9)
    first = layer(torch, ctx, s).clone()
    for _ in range(5):
        assert torch.equal(layer(torch, ctx, s), first)


def test_another_device_than_the_current(env):
    torch, fp, ctx = env
    if torch.cuda.device_count() < 2:
        pytest.skip("one GPU")
    with torch.cuda.device(1):
        x = torch.randn(4, 32, device="cuda:0")
        q, s = torch.empty(4, 32, dtype=torch.int8, device="cuda:0"), torch.empty(4, device="cuda:0")
        ctx.quantize_rows(x, q, s)
        assert torch.cuda.current_device() == 1
        assert np.array_equal(q.cpu().numpy(), quantized(x.double().cpu().numpy())[0])


# ---- the two ways of a call: the compiled binding, and the methods' own checks and conversions -----------

def unbound(fp, monkeypatch):
    monkeypatch.setattr(fp, "_bound", fp._Unbound)


@pytest.mark.parametrize("T,k,E,d,F", [(1, 2, 4, 64, 96), (33, 3, 8, 100, 77)])
def test_both_ways_give_the_same(env, monkeypatch, T, k, E, d, F):
    torch, fp, ctx = env

    def run():
        s = layer_state(torch, T, k, E, d, F, 3 * T)
        layer(torch, ctx, s)
        s["x_rows"] = torch.zeros(T * k, d, dtype=torch.bfloat16, device="cuda")
        ctx.moe_dispatch(s["x"], s["pos"], s["x_rows"])
        s["dz"], s["dw"] = torch.zeros_like(s["z"]), torch.empty_like(s["weights"])
        ctx.moe_combine_grad(s["out"], s["z"], s["pos"], s["weights"], s["dz"], s["dw"])
        s["dense"] = torch.zeros(T * k, d, device="cuda")
        ctx.matmul_i8(s["w2"][0], s["aq"], s["dense"], s["w2s"][0], s["as"])
        return s

    one = run()
    unbound(fp, monkeypatch)
    other = run()
    for name in one:
        assert name == "E" or torch.equal(one[name], other[name]), name


def test_plain_calls_go_through_the_binding(env, monkeypatch):
    torch, fp, ctx = env
    short = fp._load_binding()
    if short is fp._Unbound:
        pytest.skip("built without the compiled binding")
    seen = []

    class Watch:
        def __getattr__(self, name):
            def call(*a):
                rc = getattr(short, name)(*a)
                seen.append((name, rc))
                return rc
            return call

    monkeypatch.setattr(fp, "_bound", Watch())
    T, K, M, k, E = 5, 40, 24, 2, 4
    x = torch.randn(T, K, device="cuda")
    wide_q = torch.zeros(T * k, K + 8, dtype=torch.int8, device="cuda")
    q, sc = wide_q[:, :K], torch.zeros(T * k, device="cuda")
    e = torch.arange(T * k, dtype=torch.int32, device="cuda").view(T, k) % E
    off, pos = torch.zeros(E + 1, dtype=torch.int32, device="cuda"), torch.zeros_like(e)
    w = torch.ones(E, M, K, dtype=torch.int8, device="cuda")
    ws, y = torch.ones(E, M, device="cuda"), torch.zeros(T * k, M, device="cuda").half()
    out, dw, rows = torch.zeros(T, M, device="cuda"), torch.zeros(T, k, device="cuda"), torch.zeros(T * k, M, device="cuda")
    st = torch.cuda.current_stream()
    for stream in (None, st, st.cuda_stream):
        ctx.moe_sort(e, E, off, pos, stream=stream)
        ctx.quantize_rows(x, q, sc, pos=pos, stream=stream)
        ctx.matmul_i8(w, q, y, ws, sc, offsets=off, stream=stream)
        ctx.matmul_i8(w[1], q, y, ws[1], sc, stream=stream)
        ctx.moe_dispatch(out, pos, rows, stream=stream)
        ctx.moe_combine(y, pos, out, stream=stream)
        ctx.moe_combine_grad(out, y, pos, dweights=dw, stream=stream)
    torch.cuda.synchronize()
    assert len(seen) == 21 and all(rc == 0 for _, rc in seen), seen

    class Sub(torch.Tensor):
        pass

    del seen[:]  # what the binding does not know goes the methods' own way
    ctx.moe_combine(y, pos, out.as_subclass(Sub))
    assert seen == [("moe_combine", None)]


@pytest.mark.parametrize("way", ["binding", "methods"])
def test_refusals_of_device_tensors(env, monkeypatch, way):
    torch, fp, ctx = env
    if way == "methods":
        unbound(fp, monkeypatch)
    T, K, M, k, E = 4, 32, 16, 2, 4
    x, q, sc = torch.ones(T, K, device="cuda"), torch.zeros(T, K, dtype=torch.int8, device="cuda"), torch.ones(T, device="cuda")
    w, ws, y = torch.zeros(M, K, dtype=torch.int8, device="cuda"), torch.ones(M, device="cuda"), torch.zeros(T, M, device="cuda")
    e = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    off, pos = torch.zeros(E + 1, dtype=torch.int32, device="cuda"), torch.zeros_like(e)
    rows, wt = torch.zeros(T * k, K, device="cuda"), torch.ones(T, k, device="cuda")
    cases = [
        (lambda: ctx.quantize_rows(x.double(), q, sc), "x must be float32"),
        (lambda: ctx.quantize_rows(x.cpu(), q, sc), "x must be on cuda:0"),
        (lambda: ctx.quantize_rows(x, q[:, 1:], sc), "q must be"),
        (lambda: ctx.quantize_rows(x, q, sc[1:]), "scale must be"),
        (lambda: ctx.quantize_rows(x, q, sc.double()), "scale must be float32"),
        (lambda: ctx.quantize_rows(x.t(), q, sc), "rows must be contiguous"),
        (lambda: ctx.quantize_rows(x, q, sc, pos=pos[1:]), "pos must be"),
        (lambda: ctx.quantize_rows(x, q, sc, pos=pos.long()), "pos must be int32"),
        (lambda: ctx.matmul_i8(w, q[:, :8], y, ws, sc), "x must be"),
        (lambda: ctx.matmul_i8(w, q, y[:, :8], ws, sc), "y must be"),
        (lambda: ctx.matmul_i8(w, q, y.int(), ws, sc), "y must be float32"),
        (lambda: ctx.matmul_i8(w, q, y, ws[1:], sc), "w_scale must be"),
        (lambda: ctx.matmul_i8(w, q, y, ws, sc[1:]), "x_scale must be"),
        (lambda: ctx.matmul_i8(w[None], q, y, ws[None], sc, offsets=off), "offsets must be"),
        (lambda: ctx.matmul_i8(w, q, y, ws, sc, offsets=off), "w must be"),
        (lambda: ctx.moe_sort(e, E + 1, off, pos), "offsets must be"),
        (lambda: ctx.moe_sort(e.t(), E, off, pos.t()), "e must be contiguous"),
        (lambda: ctx.moe_sort(e, E, off, pos[1:]), "pos must be"),
        (lambda: ctx.moe_dispatch(x, pos, rows.half()), "rows must be float32"),
        (lambda: ctx.moe_dispatch(x, pos[1:], rows), "pos must be"),
        (lambda: ctx.moe_combine(rows, pos, x[:, 1:]), "out must be"),
        (lambda: ctx.moe_combine(rows, pos, x, weights=wt.half()), "weights must be float32"),
        (lambda: ctx.moe_combine(rows, pos, x, base=x.half()), "base must be float32"),
        (lambda: ctx.moe_combine_grad(x, rows[:, 1:], pos), "rows must be"),
        (lambda: ctx.moe_combine_grad(x, rows, pos, wt, drows=rows[1:]), "drows must be"),
        (lambda: ctx.moe_combine_grad(x, rows, pos, wt, dweights=wt[:, :1]), "dweights must be"),
    ]
    for call, text in cases:
        with pytest.raises(ValueError, match=text):
            call()
    # the C call's own errors come through both ways
    with pytest.raises(fp.FpError, match="fp_moe_sort") as err:
        ctx.moe_sort(e, 5000, torch.zeros(5001, dtype=torch.int32, device="cuda"), pos)
    assert err.value.code == -2


# ---- long rows of odd widths, addresses and pitches -----------------------------------------------------

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,K,pad,lead", [(300, 0, 2049, 0, 0), (150, 1, 5121, 3, 1), (300, 3, 1000, 5, 3), (20, 2, 40001, 1, 0), (33, 1, 16385, 0, 0),
                                            (33, 1, 16391, 2, 1), (40, 2, 8193, 0, 2), (33, 1, 16384, 3, 0), (500, 1, 531, 0, 0)])
def test_quantize_odd_rows(env, dtype, T, k, K, pad, lead):
    # to several rows each; rows whose maximum is a multiple of 127 (ties in every type), rows of zeros, of the type's
    # smallest values, with an infinity or a NaN at either end
    torch, fp, ctx = env
    dt = getattr(torch, dtype)
    rng = np.random.default_rng(K)
    v = rng.standard_normal((T, K)) * np.exp(rng.standard_normal((T, 1)))
    for t in range(0, T, 4):  # the halves of 127 x / a, exactly
        v[t] = np.ldexp(rng.integers(-127, 127, K) + 0.5, int(rng.integers(-6, 6)))
        v[t, rng.integers(K)] = np.ldexp(127.0, int(np.ceil(np.log2(np.abs(v[t]).max() / 127))))
    v[1], v[2] = 0.0, float(torch.finfo(dt).smallest_normal) * rng.integers(-8, 8, K) / 8
    v[3, K - 1], v[5, 0], v[6, K - 1] = math.nan, math.inf, -300.0
    x, _ = wide(torch, T, K, pad, dt, lead)
    x.copy_(torch.from_numpy(v).to(dt).cuda())
    n = T * max(k, 1) + 2
    q, qb = wide(torch, n, K, pad, torch.int8, lead)
    before, scale = qb.clone(), torch.full((n,), 5.0, device="cuda")
    pos = routed(rng, T, k, 4) if k else np.arange(T, dtype=np.int32)[:, None]
    ctx.quantize_rows(x, q, scale, pos=torch.from_numpy(pos).cuda() if k else None)
    wq, ws = quantized(x.double().cpu().numpy())
    want, wscale = np.full((n, K), 7, dtype=np.int8), np.full(n, 5.0, dtype=np.float32)
    for t in range(T):
        for p in pos[t]:
            if p >= 0:
                want[p], wscale[p] = wq[t], ws[t]
    assert np.array_equal(q.cpu().numpy(), want)
    assert np.array_equal(scale.cpu().numpy(), wscale, equal_nan=True)
    untouched(torch, q, qb, before)


@pytest.mark.parametrize("dtype,T,k,K,pad,lead", [("int8", 500, 3, 1500, 0, 5), ("int8", 3, 64, 20001, 0, 0), ("bfloat16", 300, 2, 2049, 3, 1),
                                                  ("float16", 600, 1, 2049, 1, 0), ("float32", 100, 3, 2049, 2, 1), ("int8", 1200, 2, 1025, 0, 0),
                                                  ("float32", 2, 40, 30001, 0, 3)])
def test_dispatch_odd_rows(env, dtype, T, k, K, pad, lead):
    test_moe_dispatch(env, dtype, K, pad, lead, T, k)


@pytest.mark.parametrize("rt,ot", [("bfloat16", "bfloat16"), ("float16", "float32"), ("bfloat16", "float16")])
@pytest.mark.parametrize("T,k,M,pad,lead", [(260, 3, 4099, 0, 0), (260, 1, 4099, 3, 1), (600, 2, 2055, 1, 3), (130, 5, 8192, 2, 0)])
@pytest.mark.parametrize("weighted,based", [(True, True), (False, False)])
def test_combine_odd_rows(env, rt, ot, T, k, M, pad, lead, weighted, based):
    test_moe_combine(env, rt, ot, T, k, M, pad, lead, weighted, based)


@pytest.mark.parametrize("rt,ot", [("bfloat16", "bfloat16"), ("float16", "float32"), ("bfloat16", "float16"), ("float32", "float32")])
@pytest.mark.parametrize("T,k,M,pad,lead", [(64, 3, 1501, 3, 1), (700, 2, 301, 0, 0), (3, 9, 4099, 0, 0), (900, 1, 607, 2, 5), (5, 2, 9001, 1, 0)])
def test_grad_odd_rows(env, rt, ot, T, k, M, pad, lead):
    test_moe_combine_grad(env, rt, ot, T, k, M, pad, lead)


@pytest.mark.parametrize("rt", TYPES)
@pytest.mark.parametrize("T,k,M,pad", [(40, 3, 1501, 0), (700, 2, 304, 3), (9, 2, 100, 0)])
def test_grad_parts_are_the_whole(env, rt, T, k, M, pad):
    # one gradient alone has the bits that it has beside the other, at any address of the other
    torch, fp, ctx = env
    rng = np.random.default_rng(M)
    dt = getattr(torch, rt)

    def rows(n, lead=0):
        return wide(torch, n, M, pad, dt, lead)[0]

    r, g, p = rows(T * k), rows(T), torch.from_numpy(routed(rng, T, k, 4)).cuda()
    r.copy_(torch.from_numpy(rng.standard_normal(r.shape)).cuda())
    g.copy_(torch.from_numpy(rng.standard_normal(g.shape)).cuda())
    w = torch.rand(T, k, device="cuda")
    dr, dw = rows(T * k), torch.empty(T, k, device="cuda")
    ctx.moe_combine_grad(g, r, p, w, dr, dw)
    alone, dw2, dw3 = rows(T * k, 1), torch.empty_like(dw), torch.empty_like(dw)
    ctx.moe_combine_grad(g, r, p, w, alone)
    ctx.moe_combine_grad(g, r, p, w, None, dw2)
    other = rows(T * k, 3)
    ctx.moe_combine_grad(g, r, p, w, other, dw3)
    assert torch.equal(alone, dr) and torch.equal(other, dr) and torch.equal(dw2, dw) and torch.equal(dw3, dw)


@pytest.mark.parametrize("T,K", [(3, 64), (200, 1001), (2000, 5120)])
def test_calls_follow_one_another(env, T, K):
    # kernels come onto the SMs before the one in front of them has ended, and read and write only after it: the same
    # buffers written, read and written again by calls and by torch, without a wait in between
    torch, fp, ctx = env
    k, E, n = 2, 4, 24
    g = torch.Generator(device="cuda").manual_seed(T)
    src = [torch.randn(T, K, generator=g, device="cuda").bfloat16() for _ in range(4)]
    e = [torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32) for _ in range(3)]
    w = torch.rand(T, k, generator=g, device="cuda")

    def run(wait):
        x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
        off, pos = torch.zeros(E + 1, dtype=torch.int32, device="cuda"), torch.zeros(T, k, dtype=torch.int32, device="cuda")
        rows, q, sc = torch.zeros(T * k, K, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, K, dtype=torch.int8, device="cuda"), torch.zeros(T, device="cuda")
        out, dw, dr = torch.zeros_like(x), torch.zeros(T, k, device="cuda"), torch.zeros_like(rows)
        kept = []
        torch.cuda.synchronize()
        for i in range(n):
            for call in (lambda: x.copy_(src[i % 4]),
                         lambda: ctx.moe_sort(e[i % 3], E, off, pos),
                         lambda: ctx.moe_dispatch(x, pos, rows),
                         lambda: ctx.moe_combine(rows, pos, x, weights=w, base=x),
                         lambda: ctx.quantize_rows(x, q, sc),
                         lambda: ctx.moe_sort(e[(i + 1) % 3], E, off, pos),
                         lambda: ctx.moe_combine_grad(x, rows, pos, w, dr, dw),
                         lambda: ctx.moe_dispatch(x, pos, rows),
                         lambda: ctx.moe_combine(dr, pos, out),
                         lambda: kept.append([t.clone() for t in (q, sc, out, dw, rows)]) if i % 8 == 7 else None):
                call()
                if wait:
                    torch.cuda.synchronize()
        return kept

    for one, other in zip(run(True), run(False)):
        for a, b in zip(one, other):
            assert torch.equal(a, b)


# ---- products of many tiles: blocks that take several, one after the other -----------------------------

def ragged(n, lo, hi, seed, empty=0.0):
    """n groups of lo to hi rows, some of them without any."""
    rng = np.random.default_rng(seed)
    return [int(c) for c in rng.integers(lo, hi + 1, n) * (rng.random(n) >= empty)]


# tokens or groups, channels, K, pitches beyond the row (x, y)
MANY_TILES = {
    # pairs of blocks, 256 channels by 256 tokens: the last channel tile is the first block's alone, the last tokens are no
    # multiple of 32
    "pairs": (700, 6000, 640, 0, 0),
    "pairs, odd rows of y": (603, 6001, 768, 16, 3),
    "pairs, long K": (900, 5000, 2048, 0, 8),
    "pairs, ragged groups": ([300, 1, 0, 64, 513, 33, 257, 340, 65, 0], 2500, 1536, 0, 0),
    "pairs, groups of up to 64": (ragged(40, 36, 64, 1), 1500, 1536, 0, 0),
    "pairs, odd pitches": ([500, 64, 1, 535], 2000, 1541, 3, 5),
    # tiles of 128 tokens, with main loops of a single k-tile
    "128, groups of up to 64, short K": (ragged(64, 33, 64, 2), 600, 128, 0, 0),
    "128, all sizes, short K": (ragged(40, 0, 300, 3, 0.2), 900, 112, 0, 4),
    "128, one group": (4000, 2050, 100, 12, 0),
    # tiles of 32
    "32, groups of up to 16": (ragged(100, 0, 16, 4), 1000, 128, 0, 0),
    "32, groups of up to 16, long K": (ragged(60, 1, 16, 5), 700, 2064, 0, 1),
    # weights read by classes of rows
    "classes, short K": (ragged(30, 1, 60, 6), 2500, 65, 0, 0),
    "classes, two of them": (ragged(30, 20, 64, 7), 2000, 520, 0, 3),
}


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name", MANY_TILES)
def test_matmul_many_tiles(env, name, dtype):
    # small tiles alternate between the two halves of a block's epilogue; a sum's bits hang on nothing but the inputs
    torch, fp, ctx = env
    counts, M, K, padx, pady = MANY_TILES[name]
    E, ends, off = 0, None, None
    N = counts
    if not isinstance(counts, int):
        E, N, ends = len(counts), sum(counts) + 2, np.concatenate([[0], np.cumsum(counts)])
        off = torch.from_numpy(ends.astype(np.int32)).cuda()
    w, x, ws, xs, y, yb = product_case(torch, N, M, K, E, dtype, 7 * M + K, padx=padx, pady=pady)
    y.fill_(7)
    before = yb.clone()
    ctx.matmul_i8(w, x, y, ws, xs, offsets=off)
    check_product(torch, w, x, ws, xs, y, ends)
    if E:
        assert bool((y[N - 2:] == 7).all())
    untouched(torch, y, yb, before)
    first = y.clone()
    for _ in range(8):
        y.fill_(7)
        ctx.matmul_i8(w, x, y, ws, xs, offsets=off)
        assert torch.equal(y, first)


@pytest.mark.parametrize("T,k,E,K,M", [(1400, 1, 8, 1024, 2500), (2000, 1, 40, 1536, 1500), (1200, 2, 64, 128, 600), (20, 3, 40, 256, 900),
                                       (300, 2, 30, 520, 1301), (3, 1, 1, 4096, 640)])
def test_products_follow_other_calls(env, T, k, E, K, M):
    # activations quantised, multiplied and combined over and over into the same buffers, without a wait in between
    torch, fp, ctx = env
    g = torch.Generator(device="cuda").manual_seed(T + M)
    src = [torch.randn(T, K, generator=g, device="cuda").bfloat16() for _ in range(3)]
    e = [torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32) for _ in range(2)]
    w = torch.randint(-128, 128, (E, M, K), generator=g, device="cuda", dtype=torch.int8)
    ws, wt = torch.rand(E, M, generator=g, device="cuda") * 1e-3, torch.rand(T, k, generator=g, device="cuda")

    def run(wait):
        x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
        off, pos = torch.zeros(E + 1, dtype=torch.int32, device="cuda"), torch.zeros(T, k, dtype=torch.int32, device="cuda")
        q, sc = torch.zeros(T * k, K, dtype=torch.int8, device="cuda"), torch.zeros(T * k, device="cuda")
        y, out = torch.zeros(T * k, M, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, M, device="cuda")
        kept = []
        torch.cuda.synchronize()
        for i in range(12):
            for call in (lambda: x.copy_(src[i % 3]),
                         lambda: ctx.moe_sort(e[i % 2], E, off, pos),
                         lambda: ctx.quantize_rows(x, q, sc, pos=pos),
                         lambda: ctx.matmul_i8(w, q, y, ws, sc, offsets=off),
                         lambda: ctx.moe_combine(y, pos, out, weights=wt),
                         lambda: ctx.matmul_i8(w, q, y, ws, sc, offsets=off),
                         lambda: ctx.moe_combine(y, pos, out, weights=wt, base=out),
                         lambda: y.zero_(),
                         lambda: kept.append(out.clone()) if i % 4 == 3 else None):
                call()
                if wait:
                    torch.cuda.synchronize()
        return kept

    for a, b in zip(run(True), run(False)):
        assert bool(a.any()) and torch.equal(a, b)


# ---- a bounded wait that ran out ------------------------------------------------------------------------

@pytest.mark.parametrize("way", ["binding", "methods"])
def test_a_wait_that_ran_out_is_reported_once(env, monkeypatch, way):
    # by whichever call comes next, which then queues nothing, or by the status; the context stays usable
    torch, fp, _ = env
    if way == "methods":
        unbound(fp, monkeypatch)
    ctx = fp.Context(0)
    try:
        T, k, K, M, E = 6, 2, 32, 24, 3
        x, out = torch.randn(T, K, device="cuda"), torch.zeros(T, M, device="cuda")
        e = torch.randint(0, E, (T, k), device="cuda", dtype=torch.int32)
        off, pos = torch.zeros(E + 1, dtype=torch.int32, device="cuda"), torch.zeros_like(e)
        q, s = torch.zeros(T * k, K, dtype=torch.int8, device="cuda"), torch.zeros(T * k, device="cuda")
        rows, y = torch.zeros(T * k, K, device="cuda"), torch.zeros(T * k, M, device="cuda")
        w, ws = torch.ones(E, M, K, dtype=torch.int8, device="cuda"), torch.ones(E, M, device="cuda")
        dw = torch.zeros(T, k, device="cuda")
        calls = [(off, lambda: ctx.moe_sort(e, E, off, pos)), (q, lambda: ctx.quantize_rows(x, q, s, pos=pos)),
                 (rows, lambda: ctx.moe_dispatch(x, pos, rows)), (y, lambda: ctx.matmul_i8(w, q, y, ws, s, offsets=off)),
                 (out, lambda: ctx.moe_combine(y, pos, out)), (dw, lambda: ctx.moe_combine_grad(out, y, pos, dweights=dw)),
                 (None, ctx.ops_status), (None, ctx.ops_selftest)]
        ctx.ops_status()
        for written, call in calls:
            before = None if written is None else written.clone()
            ctx.ops_selftest()
            torch.cuda.synchronize()
            with pytest.raises(fp.FpError, match="ran out") as err:
                call()
            assert err.value.code == -4
            torch.cuda.synchronize()
            assert before is None or torch.equal(written, before)
            ctx.ops_status()
            if call != ctx.ops_selftest:
                call()
        torch.cuda.synchronize()
        assert bool(out.any())
        # a captured one is reported after the replay, and again after the next
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ctx.ops_selftest()
        ctx.ops_status()
        for _ in range(2):
            g.replay()
            torch.cuda.synchronize()
            with pytest.raises(fp.FpError):
                ctx.ops_status()
            ctx.ops_status()
        del g
    finally:
        ctx.close()


@pytest.mark.parametrize("way", ["binding", "methods"])
def test_views_still_to_be_conjugated_or_negated(env, monkeypatch, way):
    torch, fp, ctx = env
    if way == "methods":
        unbound(fp, monkeypatch)
    z = torch.randn(4, 8, dtype=torch.complex64, device="cuda")
    pos, rows = torch.arange(4, dtype=torch.int32, device="cuda")[:, None], torch.zeros_like(z)
    neg = torch._neg_view(z.real.contiguous())
    q, s = torch.zeros(4, 8, dtype=torch.int8, device="cuda"), torch.zeros(4, device="cuda")
    for call in (lambda: ctx.moe_dispatch(z.conj(), pos, rows), lambda: ctx.moe_dispatch(z, pos, rows.conj()),
                 lambda: ctx.quantize_rows(neg, q, s), lambda: ctx.quantize_rows(neg.resolve_neg(), q, torch._neg_view(s)),
                 lambda: ctx.moe_combine(neg, pos, z.real.contiguous())):
        with pytest.raises(ValueError, match="resolved"):
            call()
    ctx.moe_dispatch(z.conj().resolve_conj(), pos, rows)
    assert torch.equal(rows, z.conj())
    ctx.quantize_rows(neg.resolve_neg(), q, s)
    assert np.array_equal(q.cpu().numpy(), quantized(-z.real.double().cpu().numpy())[0])


def test_earlier_errors_are_not_the_operators(env):
    # a context for a device that is not there leaves an error behind; calls that are queued do not report it
    torch, fp, ctx = env
    x, pos = torch.randn(5, 32, device="cuda"), torch.arange(5, dtype=torch.int32, device="cuda")[:, None]
    q, s, rows, out = torch.zeros(5, 32, dtype=torch.int8, device="cuda"), torch.zeros(5, device="cuda"), torch.zeros_like(x), torch.zeros_like(x)
    dw, w, y = torch.zeros(5, 1, device="cuda"), torch.ones(7, 32, dtype=torch.int8, device="cuda"), torch.zeros(5, 7, device="cuda")
    for call in (lambda: ctx.quantize_rows(x, q, s), lambda: ctx.moe_dispatch(x, pos, rows), lambda: ctx.moe_combine(rows, pos, out),
                 lambda: ctx.moe_combine_grad(x, rows, pos, dweights=dw), lambda: ctx.matmul_i8(w, q, y, torch.ones(7, device="cuda"), s),
                 lambda: ctx.moe_sort(pos, 4, pos.new_zeros(5), pos.new_zeros(5, 1))):
        with pytest.raises(fp.FpError):
            fp.Context(1000)
        call()
    assert torch.equal(rows, x) and torch.equal(out, x)


@pytest.mark.parametrize("K", [64, 77])
def test_matmul_offsets_past_the_rows(env, K):
    # every offset counts as the largest up to it, inside [0, N]; nothing behind the last row is written
    torch, fp, ctx = env
    for off, ends in (([-5, 3, 2, 30, 2 ** 31 - 1], [0, 3, 3, 20, 20]), ([-2 ** 31, -1, 0, 20, 21], [0, 0, 0, 20, 20]),
                      ([2, 5, 5, 9, 99], [2, 5, 5, 9, 20]), ([21, 25, 0, 7, 20], [20, 20, 20, 20, 20])):
        w, x, ws, xs, whole, yb = product_case(torch, 24, 40, K, 4, "float32", 3, pady=3)
        y = whole[:20]
        whole.fill_(7)
        before = yb.clone()
        ctx.matmul_i8(w, x[:20], y, ws, xs[:20], offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
        check_product(torch, w, x[:20], ws, xs[:20], y, ends)
        assert bool((y[:ends[0]] == 7).all()) and bool((y[ends[-1]:] == 7).all())
        untouched(torch, y, yb, before)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,M,K", [(96, 6000, 4096), (128, 4096, 8192), (200, 2900, 2048), (127, 6001, 1665)])
def test_matmul_split_sums_of_many_tokens(env, dtype, N, M, K):
    # tiles of 128 tokens with K split among the blocks of a cluster
    torch, fp, ctx = env
    w, x, ws, xs, y, yb = product_case(torch, N, M, K, 0, dtype, N + M, padx=16, pady=1)
    before = yb.clone()
    ctx.matmul_i8(w, x, y, ws, xs)
    check_product(torch, w, x, ws, xs, y)
    untouched(torch, y, yb, before)


def test_memory_of_odd_pitches_is_given_back(env):
    # the copies of 4 x 8192 rows of 8193 bytes, 270 MB, are kept for later calls until they are trimmed
    torch, fp, _ = env
    ctx = fp.Context(0)
    try:
        E, M, K, counts = 4, 8192, 8193, [300, 0, 250, 50]
        ends = np.concatenate([[0], np.cumsum(counts)])
        w, x, ws, xs, y, yb = product_case(torch, 600, M, K, E, "bfloat16", 21)
        off, want = torch.from_numpy(ends.astype(np.int32)).cuda(), torch.empty_like(y)

        def taken():
            torch.cuda.synchronize()
            return free - torch.cuda.mem_get_info(0)[0]

        ctx.matmul_i8(w[:, :, :K - 1].contiguous(), x[:, :K - 1].contiguous(), want, ws, xs, offsets=off)  # (loads the kernels)
        ctx.matmul_i8(w[0, :64], x[:3], y[:3, :64], ws[0, :64], xs[:3])
        torch.cuda.synchronize()
        ctx.ops_trim()
        torch.cuda.empty_cache()
        torch.cuda.synchronize()
        free = torch.cuda.mem_get_info(0)[0]
        for _ in range(2):
            y.zero_()
            ctx.matmul_i8(w, x, y, ws, xs, offsets=off)
            assert taken() >= E * M * K
            ctx.ops_trim()
            assert taken() < E * M * K // 8
        check_product(torch, w[:, :300], x, ws[:, :300], xs, y[:, :300], ends)
    finally:
        ctx.close()


@pytest.mark.parametrize("captured", [False, True])
def test_joined_streams(env, captured):
    # a base made on a second stream, waited for between two calls of the first: neither starts before what it waits for
    torch, fp, ctx = env
    T, k, E, K, M = 700, 2, 8, 512, 4096
    g = torch.Generator(device="cuda").manual_seed(2)
    x, e = torch.randn(T, K, generator=g, device="cuda"), torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    w = torch.randint(-128, 128, (E, M, K), generator=g, device="cuda", dtype=torch.int8)
    ws, wt = torch.rand(E, M, generator=g, device="cuda") * 1e-3, torch.rand(T, k, generator=g, device="cuda")
    a, b = (torch.randn(M, M, generator=g, device="cuda") for _ in range(2))
    off, pos = torch.zeros(E + 1, dtype=torch.int32, device="cuda"), torch.zeros(T, k, dtype=torch.int32, device="cuda")
    q, s, y = torch.zeros(T * k, K, dtype=torch.int8, device="cuda"), torch.zeros(T * k, device="cuda"), torch.zeros(T * k, M, device="cuda")
    base, out, back = torch.zeros(T, M, device="cuda"), torch.zeros(T, M, device="cuda"), torch.zeros(T, M, device="cuda")
    main, side = torch.cuda.Stream(), torch.cuda.Stream()

    def work(together):
        other = side if together else main
        other.wait_stream(main)
        with torch.cuda.stream(other):
            torch.mm(a[:T], b, out=base)  # takes longer than what the first stream has meanwhile
            base.add_(1.0)
        with torch.cuda.stream(main):
            ctx.moe_sort(e, E, off, pos)
            ctx.quantize_rows(x, q, s, pos=pos)
            ctx.matmul_i8(w, q, y, ws, s, offsets=off)
            main.wait_stream(other)
            ctx.moe_combine(y, pos, out, weights=wt, base=base)
        other.wait_stream(main)
        with torch.cuda.stream(other):
            ctx.moe_combine(y, pos, back, base=out)
            base.zero_()
        main.wait_stream(other)
        with torch.cuda.stream(main):
            ctx.moe_sort(e, E, off, pos)

    work(False)
    torch.cuda.synchronize()
    want, wanted = out.clone(), back.clone()
    run = lambda: work(True)  # noqa: E731
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=main):
            work(True)
        run = graph.replay
    for _ in range(5):
        y.zero_(), out.zero_(), back.zero_(), pos.zero_(), off.zero_()
        torch.cuda.synchronize()
        run()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(back, wanted)
