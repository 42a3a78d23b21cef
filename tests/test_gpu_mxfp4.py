"""GPU parity of the MXFP4 operators against the CPU oracle (needs an MI355X).

Bars: codes, scale bytes and read-back values equal; products within the
bound oracle.mxfp4 derives for fp32 accumulation in any order; sums that are
exact in fp32 equal.
"""
import numpy as np
import pytest

import workloads as W
from oracle import kquant, mxfp4

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def rz():
    import fp8_prefill_gemm_amd as rz
    rz.lib()  # loud failure if the HIP library is missing
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return rz


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def same(got, want):
    assert np.array_equal(host(got), want)


def random_tensor(seed, rows, k, spread=0):
    """(codes, bytes) with every nibble, scales 2^-spread .. 2^spread."""
    g = W.rng(seed)
    return (g.integers(0, 16, (rows, k)).astype(np.uint8),
            g.integers(127 - spread, 128 + spread, (rows, k // 32)).astype(np.uint8))


def tiled(t):
    return tuple(dev(x) for x in mxfp4.tile(*t))


def within(y, ref, bound):
    err = np.abs(host(y).astype(np.float64) - ref)
    bad = ~(err <= bound)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.size} outside the bound; first at {np.argwhere(bad)[0]}, "
                           f"err {err[bad][0]:.3g} > {np.broadcast_to(bound, err.shape)[bad][0]:.3g}")


# ---------------------------------------------------------------- quantisation

@pytest.mark.parametrize("m,k", [(1, 256), (5, 512), (32, 256), (33, 768), (64, 3584), (257, 1024)])
def test_quant(rz, m, k):
    x = W.act_normal(100 + m + k, m, k)
    x[:, :8] *= 50
    codes, scales = rz.rz_mxfp4_quant(dev(x))
    tc, ts = mxfp4.quant_tiled(x)
    same(codes, tc)
    same(scales, ts)


def test_quant_every_boundary(rz):
    """Each E2M1 rounding border, one float either side, at scales across the whole range,
    signs, zeros, subnormals, the largest finite value, infinities and NaN."""
    near = []
    for v in [0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, 7.0]:
        f = np.float32(v)
        near += [f, np.nextafter(f, np.float32(9)), np.nextafter(f, np.float32(-9))]
    near = np.array(near, dtype=np.float32)  # 48 values around X = 1
    near = np.concatenate([near, -near])
    rows = []
    for e in list(range(-149, 126, 7)) + [-127, -126, -125, -124, 124, 125]:
        for part in range(4):
            b = np.zeros(32, dtype=np.float64)
            b[:24] = near[24 * part:24 * part + 24]
            b[24] = 4.0
            rows.append(np.ldexp(b, e).astype(np.float32))
    f = np.finfo(np.float32)
    for s in ([f.max, -f.max, 1.0], [np.inf, 1.0], [1.0, -np.inf], [np.nan], [f.tiny, -f.tiny / 2], [2.0 ** -149], [-0.0], [0.0],
              [np.nan, np.inf]):
        b = np.zeros(32, dtype=np.float32)
        b[3:3 + len(s)] = s
        rows.append(b)
    x = np.concatenate(rows)
    x = np.concatenate([x, np.zeros(-x.size % 512, dtype=np.float32)]).reshape(-1, 512)
    codes, scales = rz.rz_mxfp4_quant(dev(x))
    tc, ts = mxfp4.quant_tiled(x)
    same(scales, ts)
    same(codes, tc)


def test_quant_random_bits(rz):
    """Blocks of any finite fp32 bit patterns near one exponent."""
    g = W.rng(11)
    e = g.integers(0, 250, (256, 16)).repeat(32, axis=1)
    bits = (g.integers(0, 2, e.shape) << 31) | (np.maximum(e - g.integers(0, 6, e.shape), 0) << 23) | g.integers(0, 1 << 23, e.shape)
    x = bits.astype(np.uint32).view(np.float32)
    codes, scales = rz.rz_mxfp4_quant(dev(x))
    tc, ts = mxfp4.quant_tiled(x)
    same(scales, ts)
    same(codes, tc)


@pytest.mark.parametrize("qtype", [W.Q4_K, W.Q6_K])
@pytest.mark.parametrize("n,k", [(1, 256), (33, 512), (70, 2304), (512, 3584)])
def test_pack_weight(rz, qtype, n, k):
    blocks = W.weight_blocks(qtype, 200 + n, n, k)
    codes, scales = rz.rz_mxfp4_pack_weight(qtype, dev(blocks), n, k)
    tc, ts = mxfp4.quant_tiled(kquant.dequant(qtype, blocks, n, k))
    same(scales, ts)
    same(codes, tc)


@pytest.mark.parametrize("qtype,at", [(W.Q4_K, (0, 2)), (W.Q6_K, (208,))])
def test_pack_weight_special_scales(rz, qtype, at):
    """f16 block scales of zero, subnormal, largest, infinite and NaN."""
    n, k = 32, 512
    blocks = W.weight_blocks(qtype, 300, n, k).reshape(n * 2, -1)
    specials = np.array([0x0000, 0x8000, 0x0001, 0x03FF, 0x7BFF, 0x7C00, 0xFC00, 0x7E00], dtype=np.uint16).view(np.uint8).reshape(-1, 2)
    for i in range(n * 2):
        blocks[i, at[i % len(at)]:at[i % len(at)] + 2] = specials[i % 8]
    codes, scales = rz.rz_mxfp4_pack_weight(qtype, dev(blocks), n, k)
    tc, ts = mxfp4.quant_tiled(kquant.dequant(qtype, blocks, n, k))
    same(scales, ts)
    same(codes, tc)


@pytest.mark.parametrize("m,k", [(1, 256), (37, 512), (96, 768)])
def test_dequant(rz, m, k):
    """Every code at every scale byte; bf16 and fp32 exact, fp16 rounded once."""
    g = W.rng(12)
    t = (g.integers(0, 16, (m, k)).astype(np.uint8), g.integers(0, 256, (m, k // 32)).astype(np.uint8))
    ref = mxfp4.dequant(*t)
    codes, scales = tiled(t)
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        with np.errstate(over="ignore"):
            want = torch.from_numpy(ref).to(torch.float64).numpy()
            want = want.astype(np.float16) if dtype is torch.float16 else want.astype(np.float32)
        got = host(rz.rz_mxfp4_dequant(codes, scales, m, dtype=dtype).float())
        assert np.array_equal(got, want.astype(np.float32), equal_nan=True), dtype


def test_dequant_leaves_rows_behind(rz):
    t = random_tensor(13, 3, 256)
    out = torch.full((5, 256), 7.0, device="cuda")
    rz.rz_mxfp4_dequant(*tiled(t), 3, out=out[:3])
    got = host(out)
    assert np.array_equal(got[:3], mxfp4.dequant(*t)) and (got[3:] == 7).all()


# ---------------------------------------------------------------- products

SHAPES = [(1, 1, 256), (1, 33, 512), (31, 64, 768), (37, 129, 3584), (64, 32, 2304), (65, 300, 512), (128, 256, 256),
          (200, 512, 4096), (129, 70, 18944)]
# enough 32 x 32 blocks for the larger split workgroups (one K step, fewer than the waves; odd row groups) ...
MEDIUM = [(100, 2500, 1024), (70, 3300, 512), (290, 3001, 768), (97, 8100, 256), (250, 7000, 2304)]
# ... for tiles of 64 tokens: short K, ragged, odd numbers of K steps, one row group ...
LOW = [(449, 4608, 512), (513, 2050, 1280), (129, 19000, 256), (33, 18944, 2304), (64, 12000, 256), (17, 40000, 768)]
# ... of 96, 160 and 192 (long K) ...
TALL = [(1700, 4800, 512), (96, 35000, 256), (4135, 2300, 4352), (4135, 2500, 4352)]
# ... and of 128
LARGE = [(2048, 3328, 256), (1541, 4001, 768), (4097, 1500, 512), (20, 38500, 256)]


@pytest.mark.parametrize("m,n,k", SHAPES + MEDIUM + LOW + TALL + LARGE)
def test_gemm(rz, m, n, k):
    print(f"mxfp4 gemm m={m} n={n} k={k}", flush=True)
    a, w = random_tensor(1000 + m, m, k, 3), random_tensor(2000 + n, n, k, 3)
    y = torch.full((m + 1, n), 7.0, device="cuda")
    rz.rz_mxfp4_gemm(*tiled(a), m, *tiled(w), n, y=y[:m])
    within(y[:m], *mxfp4.gemm(mxfp4.dequant(*a), mxfp4.dequant(*w)))
    assert (host(y[m:]) == 7).all()


@pytest.mark.parametrize("m,n", [(5, 40), (100, 2500), (290, 3001), (450, 3001), (1700, 4801), (1541, 4001)])
def test_pad_rows_do_not_matter(rz, m, n):
    """NaN scales and random codes in the operands' pad rows: the same bits as with zeros, gated (and its MXFP4 output) too."""
    k = 512
    g = W.rng(15)

    def spoilt(t):
        rows = t[0].shape[0]
        pad = mxfp4.pad_rows(rows) - rows
        more = g.integers(0, 16, (pad, k)).astype(np.uint8), np.full((pad, k // 32), 255, dtype=np.uint8)
        return tiled((np.concatenate([t[0], more[0]]), np.concatenate([t[1], more[1]])))

    n2 = -(-n // 256) * 256
    a, w = random_tensor(16, m, k, 2), random_tensor(17, n, k, 2)
    wide = small_scale(random_tensor(18, n2, k, 2), 8)
    small = small_scale(w, 8)
    assert torch.equal(rz.rz_mxfp4_gemm(*spoilt(a), m, *spoilt(w), n), rz.rz_mxfp4_gemm(*tiled(a), m, *tiled(w), n))
    assert torch.equal(rz.rz_mxfp4_gated(*spoilt(a), m, spoilt(small), spoilt(small), n), rz.rz_mxfp4_gated(*tiled(a), m, tiled(small), tiled(small), n))
    for p, q in zip(rz.rz_mxfp4_gated_quant(*spoilt(a), m, tiled(wide), tiled(wide), n2), rz.rz_mxfp4_gated_quant(*tiled(a), m, tiled(wide), tiled(wide), n2)):
        assert torch.equal(p, q)
    x = dev(W.act_normal(19, 3, k))
    assert torch.equal(rz.rz_mxfp4_gemv(*spoilt(w), n, x), rz.rz_mxfp4_gemv(*tiled(w), n, x))
    assert torch.equal(rz.rz_mxfp4_gated_gemv(spoilt(small), spoilt(small), n, x[:1]), rz.rz_mxfp4_gated_gemv(tiled(small), tiled(small), n, x[:1]))


@pytest.mark.parametrize("m,n,k", [(40, 96, 18944), (2048, 3500, 512)])
def test_gemm_exact_sums(rz, m, n, k):
    """With one scale every sum is a multiple of 2^-2 below 2^22: exact in fp32, so equal."""
    a, w = random_tensor(3, m, k), random_tensor(4, n, k)
    y = rz.rz_mxfp4_gemm(*tiled(a), m, *tiled(w), n)
    assert np.array_equal(host(y), mxfp4.gemm(mxfp4.dequant(*a), mxfp4.dequant(*w))[0])


@pytest.mark.parametrize("m,n", [(40, 70), (1700, 4000)])
def test_gemm_scale_range_and_nan(rz, m, n):
    """Scale bytes far apart (products from 2^-120 to 2^100), zero blocks, NaN blocks in single rows."""
    k = 512
    g = W.rng(5)
    a, w = random_tensor(6, m, k), random_tensor(7, n, k)
    a[1][:] = g.integers(70, 180, a[1].shape)
    w[1][:] = g.integers(70, 180, w[1].shape)
    a[1][3, 2] = 255
    w[1][5, 9] = 255
    a[1][7], a[0][7] = 0, 0
    av, wv = mxfp4.dequant(*a), mxfp4.dequant(*w)
    ref, bound = mxfp4.gemm(np.nan_to_num(av), np.nan_to_num(wv))
    y = host(rz.rz_mxfp4_gemm(*tiled(a), m, *tiled(w), n)).astype(np.float64)
    nan = np.zeros((m, n), dtype=bool)
    nan[3], nan[:, 5] = True, True
    assert np.array_equal(np.isnan(y), nan)
    # results under the smallest normal may be flushed inside the matrix core
    assert (np.abs(y - ref)[~nan] <= bound[~nan] + 2.0 ** -126).all()
    assert (y[7][~nan[7]] == 0).all()


def test_gemm_empty(rz):
    e = (torch.empty((0, 4, 1024), dtype=torch.uint8, device="cuda"), torch.empty((0, 1, 256), dtype=torch.uint8, device="cuda"))
    t = tiled(random_tensor(8, 3, 256))
    assert rz.rz_mxfp4_gemm(*e, 0, *t, 3).shape == (0, 3)
    assert rz.rz_mxfp4_gemm(*t, 3, *e, 0).shape == (3, 0)
    assert rz.rz_mxfp4_quant(torch.empty((0, 256), device="cuda"))[0].shape == (0, 4, 1024)
    assert rz.rz_mxfp4_dequant(*e, 0).shape == (0, 256)
    assert rz.rz_mxfp4_gemv(*t, 3, torch.empty((0, 256), device="cuda")).shape == (0, 3)


def gated_ref(a, g, u):
    av = mxfp4.dequant(*a)
    return mxfp4.gated(mxfp4.gemm(av, mxfp4.dequant(*g)), mxfp4.gemm(av, mxfp4.dequant(*u)))


def small_scale(t, by):
    """Gate arguments of a few units: silu's interesting range."""
    return t[0], t[1] - np.uint8(by)


@pytest.mark.parametrize("m,n,k", [(1, 1, 256), (37, 129, 3584), (65, 300, 512), (130, 64, 2304), (300, 1000, 768), (2049, 1700, 512),
                                   (1024, 3500, 768), (7, 19300, 256), (130, 9000, 768), (65, 6100, 256),
                                   (1700, 2400, 768), (4135, 1100, 4352), (4135, 1250, 4352)])
def test_gated(rz, m, n, k):
    print(f"mxfp4 gated m={m} n={n} k={k}", flush=True)
    a, g, u = random_tensor(30 + m, m, k, 2), small_scale(random_tensor(31, n, k, 2), 8), small_scale(random_tensor(32, n, k, 2), 8)
    h = torch.full((m + 1, n), 7.0, device="cuda")
    rz.rz_mxfp4_gated(*tiled(a), m, tiled(g), tiled(u), n, h=h[:m])
    within(h[:m], *gated_ref(a, g, u))
    assert (host(h[m:]) == 7).all()


@pytest.mark.parametrize("m,n,k", [(1, 256, 256), (37, 512, 512), (100, 256, 3584), (333, 1024, 512), (200, 4608, 512), (97, 4864, 1792), (1990, 1792, 512),
                                   (1700, 2560, 768), (4135, 1024, 4352), (4135, 1280, 4352)])
def test_gated_quant_is_quant_of_gated(rz, m, n, k):
    """Codes and bytes equal those of quantising the fp32 result, pad rows included."""
    a, g, u = tiled(random_tensor(40, m, k, 2)), tiled(small_scale(random_tensor(41, n, k, 2), 8)), tiled(small_scale(random_tensor(42, n, k, 2), 8))
    hc, hs = rz.rz_mxfp4_gated_quant(*a, m, g, u, n)
    tc, ts = mxfp4.quant_tiled(host(rz.rz_mxfp4_gated(*a, m, g, u, n)))
    same(hs, ts)
    same(hc, tc)


@pytest.mark.parametrize("m,n", [(40, 256), (400, 1024), (269, 4096), (1700, 2560), (1600, 2048)])
def test_gated_quant_nan_rows(rz, m, n):
    """NaN blocks in one token and in one gate row: exactly their blocks read as NaN, the rest as without them."""
    k = 512
    a, g, u = random_tensor(43, m, k, 2), small_scale(random_tensor(44, n, k, 2), 8), small_scale(random_tensor(45, n, k, 2), 8)
    clean = host(rz.rz_mxfp4_dequant(*rz.rz_mxfp4_gated_quant(*tiled(a), m, tiled(g), tiled(u), n), m))
    a[1][33, 5] = 255
    g[1][70, 9] = 255
    hc, hs = rz.rz_mxfp4_gated_quant(*tiled(a), m, tiled(g), tiled(u), n)
    got = host(rz.rz_mxfp4_dequant(hc, hs, m))
    nan = np.zeros((m, n), dtype=bool)
    nan[33], nan[:, 64:96] = True, True
    assert np.array_equal(np.isnan(got), nan) and np.array_equal(got[~nan], clean[~nan])
    tc, ts = mxfp4.quant_tiled(host(rz.rz_mxfp4_gated(*tiled(a), m, tiled(g), tiled(u), n)))
    same(hs, ts)
    same(hc, tc)


@pytest.mark.parametrize("n,k", [(1, 256), (37, 512), (100, 3584), (64, 18944), (48, 4096), (5000, 2304)])
@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 6, 7, 8])
def test_gemv(rz, m, n, k):
    w, u = random_tensor(50, n, k, 3), small_scale(random_tensor(51, n, k, 2), 6)
    x = W.act_normal(52 + m, m, k)
    y = torch.full((m + 1, n), 7.0, device="cuda")
    rz.rz_mxfp4_gemv(*tiled(w), n, dev(x), y=y[:m])
    ry = mxfp4.gemv(x, mxfp4.dequant(*w))
    within(y[:m], *ry)
    assert (host(y[m:]) == 7).all()
    gate = small_scale(w, 6)
    h = rz.rz_mxfp4_gated_gemv(tiled(gate), tiled(u), n, dev(x))
    within(h, *mxfp4.gated(mxfp4.gemv(x, mxfp4.dequant(*gate)), mxfp4.gemv(x, mxfp4.dequant(*u))))


def test_gemv_nan_and_zero(rz):
    """A NaN weight block reaches its row alone; an all-zero token gives zeros."""
    w = random_tensor(53, 40, 512)
    w[1][6, 3] = 255
    x = W.act_normal(54, 2, 512)
    x[1] = 0
    y = host(rz.rz_mxfp4_gemv(*tiled(w), 40, dev(x)))
    assert np.isnan(y[:, 6]).all() and np.isfinite(np.delete(y, 6, 1)).all() and (np.delete(y, 6, 1)[1] == 0).all()


@pytest.mark.parametrize("m", [1, 2, 5, 8])
def test_gemv_ranges(rz, m):
    """Every scale a finite fp32 weight has (each row of w one) with inputs from 2^-95 to 2^24, values
    next to the largest float, and an infinity and a NaN in single tokens."""
    n, k = 40, 512
    g = W.rng(55)
    w = random_tensor(56, n, k)
    w[1][:] = np.linspace(0, 252, n).astype(np.uint8)[:, None]
    w[0][w[0] == 8] = 0
    wv = mxfp4.dequant(*w)
    x = W.act_normal(57, m, k)
    x = np.where(np.abs(x) < 2.0 ** -7, np.float32(1), x)
    for e in (-95, -40, 0, 24):
        xe = np.ldexp(x, e).astype(np.float32)
        ref, bound = mxfp4.gemv(xe, wv)
        y = host(rz.rz_mxfp4_gemv(*tiled(w), n, dev(xe))).astype(np.float64)
        # no partial sum can overflow (each is at most sum |x w|), and no result is next to the subnormals
        fine = (np.abs(xe.astype(np.float64)) @ np.abs(wv).T < 2.0 ** 127) & (np.abs(ref) > 1e-30)
        assert fine.any() and (np.abs(y - ref)[fine] <= bound[fine]).all(), e
    w[1][:] = 120
    wv = mxfp4.dequant(*w)
    x[0, 7] = np.finfo(np.float32).max
    within(rz.rz_mxfp4_gemv(*tiled(w), n, dev(x)), *mxfp4.gemv(x, wv))
    x[0, 7] = -np.inf
    x[m - 1, 9] = np.nan if m > 1 else x[0, 9]
    y = host(rz.rz_mxfp4_gemv(*tiled(w), n, dev(x)))
    with np.errstate(invalid="ignore"):
        lead = x[0, 7] * wv[:, 7].astype(np.float32)  # -inf, inf, or NaN where the weight is 0
    assert np.array_equal(y[0], lead, equal_nan=True)
    if m > 1:
        assert np.isnan(y[m - 1]).all()
    if m > 2:
        r, b = mxfp4.gemv(x[1:m - 1], wv)
        assert (np.abs(y[1:m - 1] - r) <= b).all()


# ---------------------------------------------------------------- used together

def test_feed_forward(rz):
    """K-quant weights -> MXFP4; input -> gated -> down, as codes throughout: each step against
    the oracle on the step's own input."""
    m, d, f = 100, 512, 1280
    bg, bu, bd = (W.weight_blocks(q, s, n, k) for q, s, n, k in ((W.Q4_K, 60, f, d), (W.Q4_K, 61, f, d), (W.Q6_K, 62, d, f)))
    x = W.act_normal(63, m, d)
    gate, up = rz.rz_mxfp4_pack_weight(W.Q4_K, dev(bg), f, d), rz.rz_mxfp4_pack_weight(W.Q4_K, dev(bu), f, d)
    down = rz.rz_mxfp4_pack_weight(W.Q6_K, dev(bd), d, f)
    a = rz.rz_mxfp4_quant(dev(x))
    h = rz.rz_mxfp4_gated_quant(*a, m, gate, up, f)
    y = rz.rz_mxfp4_gemm(*h, m, *down, d)

    q = {n: mxfp4.quant(kquant.dequant(t, b, *s)) for n, t, b, s in
         (("g", W.Q4_K, bg, (f, d)), ("u", W.Q4_K, bu, (f, d)), ("d", W.Q6_K, bd, (d, f)))}
    within(rz.rz_mxfp4_gated(*a, m, gate, up, f), *gated_ref(mxfp4.quant(x), q["g"], q["u"]))
    hv = host(rz.rz_mxfp4_dequant(*h, m)).astype(np.float64)
    within(y, *mxfp4.gemm(hv, mxfp4.dequant(*q["d"])))


def test_streams_and_repeats(rz):
    """Two streams at once, each call repeated: the same bits as alone."""
    ts = [(tiled(random_tensor(70 + i, 300, 512, 2)), tiled(random_tensor(80 + i, 4096, 512, 2))) for i in range(2)]
    alone = [host(rz.rz_mxfp4_gemm(*a, 300, *w, 4096)) for a, w in ts]
    streams = [torch.cuda.Stream() for _ in ts]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for (a, w), st in zip(ts, streams):
            got.append(rz.rz_mxfp4_gemm(*a, 300, *w, 4096, stream=st))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert np.array_equal(host(y), alone[i % 2])


def test_every_call_on_a_stream(rz):
    """Each function on a side stream, its outputs made there: the same bits as on the current one."""
    m, n, k = 70, 512, 768
    x = dev(W.act_normal(85, m, k))
    a, g, u = tiled(random_tensor(86, m, k, 2)), tiled(random_tensor(87, n, k, 2)), tiled(random_tensor(88, n, k, 2))
    blocks = dev(W.weight_blocks(W.Q6_K, 89, n, k))
    calls = [lambda **kw: rz.rz_mxfp4_quant(x, **kw), lambda **kw: rz.rz_mxfp4_pack_weight(W.Q6_K, blocks, n, k, **kw),
             lambda **kw: rz.rz_mxfp4_dequant(*a, m, dtype=torch.bfloat16, **kw), lambda **kw: rz.rz_mxfp4_gemm(*a, m, *g, n, **kw),
             lambda **kw: rz.rz_mxfp4_gated(*a, m, g, u, n, **kw), lambda **kw: rz.rz_mxfp4_gated_quant(*a, m, g, u, n, **kw),
             lambda **kw: rz.rz_mxfp4_gemv(*g, n, x[:3], **kw), lambda **kw: rz.rz_mxfp4_gated_gemv(g, u, n, x[:1], **kw)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for i, f in enumerate(calls):
        got, want = f(stream=side), f()
        torch.cuda.synchronize()
        for p, q in zip(got if isinstance(got, tuple) else (got,), want if isinstance(want, tuple) else (want,)):
            assert torch.equal(p, q), i


def test_refusals_of_the_library(rz):
    """What the binding lets through and the library refuses: RzError with its status, outputs untouched."""
    a, w = tiled(random_tensor(94, 3, 256)), tiled(random_tensor(95, 96, 256))
    with pytest.raises(rz.RzError, match="n=96 must be a multiple of 256") as e:
        rz.rz_mxfp4_gated_quant(*a, 3, w, w, 96)
    assert e.value.status == -3
    with pytest.raises(rz.RzError, match="m=9 exceeds 8"):
        rz.rz_mxfp4_gemv(*w, 96, torch.zeros((9, 256), device="cuda"))
    y = torch.full((3 * 96 + 1,), 7.0, device="cuda")
    with pytest.raises(rz.RzError, match="16-byte aligned"):
        rz.rz_mxfp4_gemm(*a, 3, *w, 96, y=y[1:].view(3, 96))
    assert (host(y) == 7).all()
    with pytest.raises(ValueError, match="one device expected"):
        rz.rz_mxfp4_gemm(a[0], a[1].cpu(), 3, *w, 96)


def test_graph_replays(rz):
    """quant, gated_quant, gemm and gemv captured; replayed on new inputs between eager calls."""
    m, d, f = 70, 512, 1024
    gate, up, down = tiled(random_tensor(90, f, d)), tiled(random_tensor(91, f, d)), tiled(random_tensor(92, d, f))
    gate, up = [(c, s - 8) for c, s in (gate, up)]
    x = torch.zeros((m, d), device="cuda")

    def block():
        h = rz.rz_mxfp4_gated_quant(*rz.rz_mxfp4_quant(x), m, gate, up, f)
        return rz.rz_mxfp4_gemm(*h, m, *down, d), rz.rz_mxfp4_gated_gemv(gate, up, f, x[:3])

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        block()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block()
    for i in range(4):
        x.copy_(dev(W.act_normal(93 + i, m, d)))
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(out, block()):
            assert torch.equal(got, want)


def test_large_offsets(rz):
    """Codes past 2^32 bytes: the last rows of a 2^33-value tensor, and its read-back."""
    rows, k = 1 << 19, 16384
    x = torch.zeros((rows, k), device="cuda")
    tail = W.act_normal(99, 40, k)
    x[-40:] = dev(tail)
    codes, scales = rz.rz_mxfp4_quant(x)
    del x
    tc, ts = mxfp4.quant_tiled(tail[-32:])
    same(codes[-1:], tc)
    same(scales[-1:], ts)
    w = tiled(random_tensor(98, 40, k))
    out = rz.rz_mxfp4_gemm(codes, scales, rows, *w, 40)
    within(out[-32:], *mxfp4.gemm(mxfp4.dequant(*mxfp4.quant(tail[-32:])), mxfp4.dequant(*random_tensor(98, 40, k))))
    assert (host(out[:8]) == 0).all()
    del out
    back = rz.rz_mxfp4_dequant(codes, scales, rows, dtype=torch.bfloat16)
    assert np.array_equal(host(back[-32:].float()), mxfp4.dequant(*mxfp4.quant(tail[-32:])))
