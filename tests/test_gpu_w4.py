"""4-bit weights on the GPU: the quantiser and the stored values bit for bit against the plain binary32 definition, the
few-token product against binary64 within the bound of its sums (w4_plain)."""
import numpy as np
import pytest
import torch

import w4_plain as P
import w8a8_smoothquant_gemm_b200 as sq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TD = {"bf16": torch.bfloat16, "f32": torch.float32}


def dev(a, dt=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dt is None else t.to(TD[dt])


def num(t):
    return t.detach().double().cpu().numpy()


def random_weight(rng, K, N, group, asym):
    """A packed weight with every code and zero point: (wq, sg, zp on the device, values)."""
    codes = rng.integers(0, 16, (N, K)).astype(np.uint8)
    G = -(-K // group)
    sg = P.bf16(rng.uniform(0.5, 2, (G, N)).astype(np.float32) * 0.01)
    zp = rng.integers(0, 16, (G, N)).astype(np.uint8) if asym else None
    wq = P.pack(codes)
    return (dev(wq), dev(sg).to(torch.bfloat16), None if zp is None else dev(zp)), P.values(wq, sg, zp, K, group)


def activations(rng, M, K, dt):
    x = rng.normal(0, 1, (M, K)).astype(np.float32)
    x[:, rng.choice(K, max(1, K // 100))] *= 50
    return P.bf16(x) if dt == "bf16" else x


def check(y, ref, bound, out):
    y = num(y)
    off = np.abs(y - ref)
    assert (off <= bound + np.abs(ref) * P.HALF_STEP[out] * (1 + 2.0 ** -8) + bound * P.HALF_STEP[out]).all(), (
        float((off - bound).max()))


# ------------------------------------------------------------------------------------------------ quantiser
@pytest.mark.parametrize("K,N,dt", [(16, 8, "bf16"), (128, 64, "bf16"), (144, 72, "bf16"), (1040, 1000, "f32"),
                                    (4096, 136, "bf16"), (208, 4, "f32"), (14336, 72, "bf16")])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("asym", [False, True])
def test_fold(K, N, dt, group, asym):
    rng = np.random.default_rng(K + N + group)
    W = rng.normal(0, 0.02, (K, N)).astype(np.float32)
    W[: min(K, 128), 1] = 0                          # all-zero groups
    W[:, 2] = np.abs(W[:, 2])                        # one-sided ones
    W[:, 3] = -np.abs(W[:, 3])
    W[::7, 0] *= 40
    W = P.bf16(W) if dt == "bf16" else W
    s = rng.uniform(0.2, 3, K).astype(np.float32)
    gamma, beta = rng.uniform(0.5, 1.5, K).astype(np.float32), rng.normal(0, 0.1, K).astype(np.float32)
    wq, sg, zp, gf, bf = sq.sq_fold_quant_weights_w4(dev(W, dt), dev(s), dev(gamma), dev(beta), group=group, asym=asym)
    codes, r_sg, r_zp = P.quantise(W, s, group, asym)
    assert np.array_equal(sg.float().cpu().numpy(), r_sg)
    assert np.array_equal(wq.cpu().numpy(), P.pack(codes))
    assert (zp is None) == (not asym)
    if asym:
        assert np.array_equal(zp.cpu().numpy(), r_zp)
    assert np.array_equal(gf.cpu().numpy(), gamma / s) and np.array_equal(bf.cpu().numpy(), beta / s)
    v = P.values(P.pack(codes), r_sg, r_zp, K, group)
    f32 = sq.sq_w4_dequant(wq, sg, zp, K=K, group=group, out_dtype=torch.float32)
    assert np.array_equal(num(f32), v)
    b16 = sq.sq_w4_dequant(wq, sg, zp, K=K, group=group)
    assert np.array_equal(num(b16), P.bf16(v.astype(np.float32)).astype(np.float64))


def test_fold_without_factors_and_with_a_padded_matrix():
    rng = np.random.default_rng(3)
    W = P.bf16(rng.normal(0, 0.02, (272, 96)).astype(np.float32))
    Wd = dev(W, "bf16")
    wide = torch.full((272, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, 16:112] = Wd
    a = sq.sq_fold_quant_weights_w4(wide[:, 16:112], group=64)
    b = sq.sq_fold_quant_weights_w4(Wd, torch.ones(272, device=DEV), group=64)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and a[2] is None and a[3] is None
    assert np.array_equal(a[0].cpu().numpy(), P.pack(P.quantise(W, None, 64, False)[0]))


@pytest.mark.parametrize("zero", range(16))
def test_fold_rounds_ties_to_even_codes_before_the_zero_point(zero):
    """A grid of step 1/16 with each zero point, and values on every half step of it."""
    W = np.zeros((64, 8), np.float32)
    W[:, :] = (np.arange(64)[:, None] % 31) * 0.5 - zero
    W = np.clip(W, -zero, 15 - zero) / 16
    wq, sg, zp, _, _ = sq.sq_fold_quant_weights_w4(dev(W), group=64, asym=True)
    codes, r_sg, r_zp = P.quantise(W, None, 64, True)
    assert (r_sg == 1 / 16).all() and (r_zp == zero).all()
    assert np.array_equal(zp.cpu().numpy(), r_zp) and np.array_equal(wq.cpu().numpy(), P.pack(codes))
    half = W * 16 % 1 == 0.5
    assert half.sum() > 100 and (codes.T[half].astype(int) - zero).astype(int).tolist() == np.clip(
        np.rint(W[half] * 16), -zero, 15 - zero).astype(int).tolist()


def test_fold_extreme_magnitudes():
    """Scales far outside the range of the shared reciprocal, and ones that round to zero."""
    rng = np.random.default_rng(4)
    W = rng.normal(0, 1, (128, 8)).astype(np.float32)
    W *= np.array([1e-44, 1e-40, 1e-36, 1e-30, 1e30, 1e36, 3e37, 1], np.float32)
    for asym in (False, True):
        wq, sg, zp, _, _ = sq.sq_fold_quant_weights_w4(dev(W), group=32, asym=asym)
        codes, r_sg, r_zp = P.quantise(W, None, 32, asym)
        assert np.array_equal(sg.float().cpu().numpy(), r_sg)
        assert np.array_equal(wq.cpu().numpy(), P.pack(codes))
        assert not asym or np.array_equal(zp.cpu().numpy(), r_zp)


def test_dequant_into_a_padded_matrix():
    rng = np.random.default_rng(5)
    (wq, sg, zp), v = random_weight(rng, 144, 9, 32, True)
    y = torch.full((10, 160), -7.0, device=DEV)
    sq.sq_w4_dequant(wq, sg, zp, K=144, group=32, y=y[:9, :144])
    assert np.array_equal(num(y[:9, :144]), v)
    assert (y[9] == -7).all() and (y[:, 144:] == -7).all()


# ------------------------------------------------------------------------------------------------ product
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 32, 33, 64, 70])
@pytest.mark.parametrize("K,N,group,asym,dt", [(16, 1, 32, False, "bf16"), (144, 17, 64, True, "bf16"),
                                               (1040, 129, 32, True, "f32"), (4096, 200, 128, False, "bf16")])
def test_gemm(M, K, N, group, asym, dt):
    rng = np.random.default_rng(M * K + N)
    (wq, sg, zp), w = random_weight(rng, K, N, group, asym)
    x = activations(rng, M, K, dt)
    ref, bound = P.product(x, w, group)
    for out in ("bf16", "f32"):
        check(sq.sq_w4_gemm(dev(x, dt), wq, sg, zp, group=group, out_dtype=TD[out]), ref, bound, out)


@pytest.mark.parametrize("M,K,N", [(1, 12288, 4096), (1, 49152, 64), (3, 133136, 40), (5, 14336, 1024), (1, 4096, 6144),
                                   (16, 14336, 300), (40, 14336, 130), (1, 256, 40000), (64, 128, 20000)])
@pytest.mark.parametrize("group,asym,dt", [(128, False, "bf16"), (32, True, "bf16"), (64, False, "f32")])
def test_gemm_sizes(M, K, N, group, asym, dt):
    """Long rows (x staged in pieces, K cut over clusters), few and many output channels."""
    rng = np.random.default_rng(M + K + N)
    (wq, sg, zp), w = random_weight(rng, K, N, group, asym)
    x = activations(rng, M, K, dt)
    ref, bound = P.product(x, w, group)
    y = sq.sq_w4_gemm(dev(x, dt), wq, sg, zp, group=group, out_dtype=torch.float32)
    check(y, ref, bound, "f32")
    assert torch.equal(y, sq.sq_w4_gemm(dev(x, dt), wq, sg, zp, group=group, out_dtype=torch.float32))


@pytest.mark.parametrize("M", [1, 2, 3, 5, 8])
@pytest.mark.parametrize("group,asym,dt", [(32, True, "bf16"), (64, False, "bf16"), (128, True, "bf16"), (128, False, "f32"),
                                           (64, True, "f32"), (32, False, "f32")])
def test_gemm_many_channels_for_few_tokens(M, group, asym, dt):
    """Many tiles to a CTA; tokens of very different magnitudes, one of them zero."""
    rng = np.random.default_rng(M + group)
    K, N = 528, 21008
    (wq, sg, zp), w = random_weight(rng, K, N, group, asym)
    x = activations(rng, M, K, dt)
    x[0] *= np.float32(2.0 ** -90)
    x[M - 1, 3] *= np.float32(2.0 ** 60)
    if M > 2:
        x[1] = 0
    ref, bound = P.product(x, w, group)
    check(sq.sq_w4_gemm(dev(x, dt), wq, sg, zp, group=group, out_dtype=torch.float32), ref, bound, "f32")


@pytest.mark.parametrize("M", [9, 16, 17, 31, 32, 33, 64, 65, 130])
@pytest.mark.parametrize("K,N,group,asym,dt", [(16, 8, 128, False, "bf16"), (128, 136, 32, True, "bf16"),
                                               (400, 128, 64, True, "bf16"), (1040, 1000, 64, False, "f32"),
                                               (2064, 4104, 128, True, "bf16"), (272, 40, 32, True, "f32"),
                                               (4096, 520, 32, True, "bf16"), (8192, 264, 128, False, "f32"),
                                               (4096, 1032, 64, True, "bf16"), (2064, 2056, 128, False, "bf16"),
                                               (4096, 2056, 128, True, "bf16"), (144, 30008, 128, True, "bf16"),
                                               (14336, 1096, 64, False, "bf16"), (4096, 1160, 128, True, "f32"),
                                               (400, 10488, 64, False, "f32"), (4112, 4104, 32, True, "f32")])
def test_gemm_for_a_batch(M, K, N, group, asym, dt):
    """Nine tokens and more, whole pieces of scales: last units of one block, last tiles of few channels, blocks of
    tokens that are not full, K over clusters."""
    rng = np.random.default_rng(M * K + N)
    (wq, sg, zp), w = random_weight(rng, K, N, group, asym)
    x = activations(rng, M, K, dt)
    ref, bound = P.product(x, w, group)
    for out in ("bf16", "f32"):
        y = sq.sq_w4_gemm(dev(x, dt), wq, sg, zp, group=group, out_dtype=TD[out])
        check(y, ref, bound, out)
        assert torch.equal(y, sq.sq_w4_gemm(dev(x, dt), wq, sg, zp, group=group, out_dtype=TD[out]))


@pytest.mark.parametrize("M", [12, 24, 48])
@pytest.mark.parametrize("K,N,group,asym,dt", [(2048, 50000, 64, True, "bf16"), (1040, 30008, 128, False, "f32"),
                                               (256, 60000, 32, False, "bf16")])
def test_gemm_for_a_batch_many_tiles(M, K, N, group, asym, dt):
    """Many tiles to a CTA: every ring, buffer and barrier goes round several times."""
    rng = np.random.default_rng(M + K + N)
    (wq, sg, zp), w = random_weight(rng, K, N, group, asym)
    x = activations(rng, M, K, dt)
    ref, bound = P.product(x, w, group)
    check(sq.sq_w4_gemm(dev(x, dt), wq, sg, zp, group=group, out_dtype=torch.float32), ref, bound, "f32")


@pytest.mark.parametrize("M", [9, 20, 64])
def test_gemm_for_a_batch_is_exact_on_integers(M):
    rng = np.random.default_rng(M)
    K, N = 1296, 3240
    codes = rng.integers(0, 16, (N, K)).astype(np.uint8)
    sg = (2.0 ** rng.integers(-3, 4, (-(-K // 64), N))).astype(np.float32)
    zp = rng.integers(0, 16, sg.shape).astype(np.uint8)
    wq = P.pack(codes)
    x = rng.integers(-8, 9, (M, K)).astype(np.float32)
    ref = x.astype(np.float64) @ P.values(wq, sg, zp, K, 64).T
    for dt in ("bf16", "f32"):
        y = sq.sq_w4_gemm(dev(x, dt), dev(wq), dev(sg).to(torch.bfloat16), dev(zp), group=64, out_dtype=torch.float32)
        assert np.array_equal(num(y), ref)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N", [264, 10504])
def test_gemm_for_a_batch_strides_infinities_and_the_rows_behind(dt, N):
    rng = np.random.default_rng(13)
    M, K = 21, 400
    codes = rng.integers(9, 16, (N, K)).astype(np.uint8)  # positive weights only
    sg = P.bf16(rng.uniform(0.5, 2, (4, N)).astype(np.float32))
    wq = P.pack(codes)
    w = P.values(wq, sg, None, K, 128)
    x = activations(rng, M, K, dt)
    x[1, 399], x[2, 0], x[4, 200] = np.inf, np.nan, -np.inf
    wide = torch.full((M + 1, K + 32), float("nan"), dtype=TD[dt], device=DEV)
    wide[:M, 16:K + 16] = dev(x, dt)
    y = torch.full((M + 2, N + 5), -7.0, device=DEV)
    sq.sq_w4_gemm(wide[:M, 16:K + 16], dev(wq), dev(sg).to(torch.bfloat16), y=y[1:M + 1, 3:N + 3])
    got = num(y[1:M + 1, 3:N + 3])
    assert (got[1] == np.inf).all() and np.isnan(got[2]).all() and (got[4] == -np.inf).all()
    rows = [m for m in range(M) if m not in (1, 2, 4)]
    ref, bound = P.product(x[rows], w, 128)
    assert (np.abs(got[rows] - ref) <= bound + np.abs(ref) * 2.0 ** -24).all()
    y[1:M + 1, 3:N + 3] = -7
    assert (y == -7).all()


def test_gemm_for_a_batch_scales_at_odd_addresses():
    """Scales and zero points that do not begin on a 16-byte boundary: the same values."""
    rng = np.random.default_rng(14)
    (wq, sg, zp), w = random_weight(rng, 528, 8008, 64, True)
    off_s = torch.empty(sg.numel() + 1, dtype=sg.dtype, device=DEV)[1:].view(sg.shape).copy_(sg)
    off_z = torch.empty(zp.numel() + 1, dtype=zp.dtype, device=DEV)[1:].view(zp.shape).copy_(zp)
    x = activations(rng, 40, 528, "bf16")
    for s, z in ((sg, zp), (off_s, off_z)):
        check(sq.sq_w4_gemm(dev(x, "bf16"), wq, s, z, group=64, out_dtype=torch.float32), *P.product(x, w, 64), "f32")


def test_gemm_for_a_batch_two_streams_and_graphs():
    rng = np.random.default_rng(15)
    (wq, sg, zp), w = random_weight(rng, 2048, 2056, 64, True)
    x = [activations(rng, m, 2048, "bf16") for m in (24, 64)]
    xd = [dev(a, "bf16") for a in x]
    want = [sq.sq_w4_gemm(a, wq, sg, zp, group=64) for a in xd]
    for a, y in zip(x, want):
        check(y, *P.product(a, w, 64), "bf16")
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ys = [torch.empty_like(y) for y in want]
    torch.cuda.synchronize()
    for _ in range(40):
        for a, st, y in zip(xd, streams, ys):
            sq.sq_w4_gemm(a, wq, sg, zp, group=64, y=y, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(y, v) for y, v in zip(ys, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for a, y in zip(xd, ys):
            sq.sq_w4_gemm(a, wq, sg, zp, group=64, y=y)
    for y in ys:
        y.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(y, v) for y, v in zip(ys, want))
    assert sq.sq_device_error() == 0


@pytest.mark.parametrize("M,N,K", [(32, 20000, 256), (64, 4096, 4096)])
def test_gemm_for_a_batch_gives_up(M, N, K):
    """Every wait runs out at once (one CTA a tile, then clusters): the kernel leaves and says so, and the next call is
    right again."""
    rng = np.random.default_rng(16)
    (wq, sg, _), w = random_weight(rng, K, N, 128, False)
    x = activations(rng, M, K, "bf16")
    xd = dev(x, "bf16")
    torch.cuda.synchronize()
    sq.sq_device_error(clear=True)
    sq.sq_set_wait_limit(0)
    try:
        sq.sq_w4_gemm(xd, wq, sg)
        assert sq.sq_device_error(clear=True) & 7
    finally:
        torch.cuda.synchronize()
        sq.sq_set_wait_limit(sq.WAIT_LIMIT_DEFAULT_NS)
        sq.sq_device_error(clear=True)
    check(sq.sq_w4_gemm(xd, wq, sg, out_dtype=torch.float32), *P.product(x, w, 128), "f32")
    assert sq.sq_device_error(clear=True) == 0


def test_gemm_many_tokens():
    rng = np.random.default_rng(6)
    (wq, sg, zp), w = random_weight(rng, 272, 100, 128, False)
    x = activations(rng, 1000, 272, "bf16")
    ref, bound = P.product(x, w, 128)
    check(sq.sq_w4_gemm(dev(x, "bf16"), wq, sg, zp), ref, bound, "bf16")


def test_gemm_strides_and_the_rows_behind():
    rng = np.random.default_rng(7)
    (wq, sg, zp), w = random_weight(rng, 272, 33, 32, True)
    x = activations(rng, 5, 272, "bf16")
    wide = torch.full((6, 304), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:5, 16:288] = dev(x, "bf16")
    y = torch.full((7, 37), -7.0, device=DEV)
    sq.sq_w4_gemm(wide[:5, 16:288], wq, sg, zp, group=32, y=y[1:6, 3:36])  # odd offset, odd leading dimension
    ref, bound = P.product(x, w, 32)
    check(y[1:6, 3:36], ref, bound, "f32")
    y[1:6, 3:36] = -7
    assert (y == -7).all()


@pytest.mark.parametrize("M,N", [(6, 77), (6, 19000), (1, 5000), (8, 24000)])
def test_gemm_is_exact_on_integers(M, N):
    """Small integers in x and power-of-two scales: every sum is exact, so every bit must agree."""
    rng = np.random.default_rng(8)
    K = 2064 if M == 6 and N == 77 else 304
    codes = rng.integers(0, 16, (N, K)).astype(np.uint8)
    sg = (2.0 ** rng.integers(-3, 4, (-(-K // 64), N))).astype(np.float32)
    zp = rng.integers(0, 16, sg.shape).astype(np.uint8)
    wq = P.pack(codes)
    x = rng.integers(-8, 9, (M, K)).astype(np.float32)
    ref = x.astype(np.float64) @ P.values(wq, sg, zp, K, 64).T
    for dt in ("bf16", "f32"):
        y = sq.sq_w4_gemm(dev(x, dt), dev(wq), dev(sg).to(torch.bfloat16), dev(zp), group=64, out_dtype=torch.float32)
        assert np.array_equal(num(y), ref)


def test_gemm_takes_binary32_inputs_whole():
    """24-bit inputs against 1-bit weights: what a product with rounded inputs would lose."""
    x = np.zeros((2, 128), np.float32)
    x[0, :3] = np.float32(1 + 2.0 ** -23), np.float32(2.0 ** -30 * (1 + 2.0 ** -23)), np.float32(-1)
    x[1, 5] = np.float32(np.pi) * np.float32(1e20)
    wq = P.pack(np.full((3, 128), 9, np.uint8))  # every value 1
    y = sq.sq_w4_gemm(dev(x), dev(wq), torch.ones(1, 3, dtype=torch.bfloat16, device=DEV), out_dtype=torch.float32)
    # within one cut of the tensor cores' adder at the largest partial sum
    assert np.abs(num(y)[0] - (2.0 ** -23 + 2.0 ** -30)).max() <= 2.0 ** -23 * 2.0 ** -1
    assert (num(y)[1] == np.float64(x[1, 5])).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N", [50, 15000])
def test_gemm_keeps_infinities_and_nan_in_their_rows(N, dt):
    rng = np.random.default_rng(9)
    (wq, sg, _), _ = random_weight(rng, 400, N, 128, False)
    codes = rng.integers(9, 16, (N, 400)).astype(np.uint8)  # positive weights only
    wq = dev(P.pack(codes))
    w = P.values(P.pack(codes), sg.float().cpu().numpy(), None, 400, 128)
    x = activations(rng, 6, 400, dt)
    x[1, 399], x[2, 0], x[4, 200] = np.inf, np.nan, -np.inf
    y = num(sq.sq_w4_gemm(dev(x, dt), wq, sg, out_dtype=torch.float32))
    assert (y[1] == np.inf).all() and np.isnan(y[2]).all() and (y[4] == -np.inf).all()
    rows = [0, 3, 5]
    ref, bound = P.product(x[rows], w, 128)
    assert (np.abs(y[rows] - ref) <= bound + np.abs(ref) * 2.0 ** -24).all()


def test_gemm_past_32_bit_offsets():
    """A packed weight of 2.4 GB: rows whose bytes lie past 2^31 and 2^32 code positions."""
    K, N = 8192, 600_000
    wq = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=DEV)
    sg = (torch.rand(K // 128, N, device=DEV) * 0.01 + 0.005).to(torch.bfloat16)
    rng = np.random.default_rng(10)
    x = activations(rng, 1, K, "bf16")
    y = sq.sq_w4_gemm(dev(x, "bf16"), wq, sg, out_dtype=torch.float32)
    rows = torch.tensor([0, 1, 300_000, 524_288, 599_998, 599_999], device=DEV)
    w = P.values(wq[rows].cpu().numpy(), sg[:, rows].float().cpu().numpy(), None, K, 128)
    ref, bound = P.product(x, w, 128)
    check(y[:, rows], ref, bound, "f32")
    part = sq.sq_w4_dequant(wq[524_288:524_296], sg[:, 524_288:524_296].contiguous(), K=K, out_dtype=torch.float32)
    assert np.array_equal(num(part), P.values(wq[524_288:524_296].cpu().numpy(),
                                              sg[:, 524_288:524_296].float().cpu().numpy(), None, K, 128))


def test_empty_calls():
    wq, sg = torch.zeros(0, 128, dtype=torch.uint8, device=DEV), torch.zeros(2, 0, dtype=torch.bfloat16, device=DEV)
    x = torch.ones(3, 256, dtype=torch.bfloat16, device=DEV)
    assert sq.sq_w4_gemm(x, wq, sg).shape == (3, 0)
    wq, sg = torch.zeros(8, 128, dtype=torch.uint8, device=DEV), torch.zeros(2, 8, dtype=torch.bfloat16, device=DEV)
    assert sq.sq_w4_gemm(x[:0], wq, sg).shape == (0, 8)


def test_gemm_on_another_stream_and_in_a_graph():
    rng = np.random.default_rng(11)
    (wq, sg, zp), w = random_weight(rng, 1024, 96, 64, True)
    xs = [activations(rng, 3, 1024, "bf16") for _ in range(3)]
    st = torch.cuda.Stream()
    x, y = dev(xs[0], "bf16"), torch.empty(3, 96, device=DEV)
    st.wait_stream(torch.cuda.current_stream())
    sq.sq_w4_gemm(x, wq, sg, zp, group=64, y=y, stream=st)
    st.synchronize()
    check(y, *P.product(xs[0], w, 64), "f32")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        sq.sq_w4_gemm(x, wq, sg, zp, group=64, y=y)
        sq.sq_w4_gemm(x, wq, sg, zp, group=64, y=y)
    for a in xs:
        x.copy_(dev(a, "bf16"))
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        check(y, *P.product(a, w, 64), "f32")


def test_a_layer_from_its_weights_to_its_output():
    """Calibration, factors, 4-bit fold, product: against the exact product with the quantised weights, and near the
    unquantised layer; the W8A8 GEMM's output feeds the 4-bit product (programmatic launches back to back)."""
    rng = np.random.default_rng(12)
    K, H, N, M = 1024, 2048, 512, 5
    x = activations(rng, M, K, "bf16")
    W1 = P.bf16(rng.normal(0, 0.03, (K, H)).astype(np.float32))
    W2 = P.bf16(rng.normal(0, 0.03, (H, N)).astype(np.float32))
    xd, W1d, W2d = dev(x, "bf16"), dev(W1, "bf16"), dev(W2, "bf16")
    s1 = sq.sq_smooth_factors(sq.sq_calib_absmax(xd, 0), sq.sq_calib_absmax(W1d, 1), 0.5)
    wq1, sw1, _, _ = sq.sq_fold_quant_weights(W1d, s1)
    wq2, sg2, zp2, _, _ = sq.sq_fold_quant_weights_w4(W2d, group=64, asym=True)
    xq, sx = sq.sq_ln_smooth_quant(xd, s=s1)
    h = sq.sq_w8a8_gemm(xq, sx, wq1, sw1)
    y = sq.sq_w4_gemm(h, wq2, sg2, zp2, group=64)
    v = P.values(wq2.cpu().numpy(), sg2.float().cpu().numpy(), zp2.cpu().numpy(), H, 64)
    check(y, *P.product(num(h), v, 64), "bf16")
    full = x.astype(np.float64) @ W1.astype(np.float64) @ W2.astype(np.float64)
    assert np.linalg.norm(num(y) - full) < 0.15 * np.linalg.norm(full)
