"""The 4-bit product on the ways that large weights take: binary32 inputs bit for bit in every kernel, several passes of
tiles, x in chunks of K; and the quantiser's scale where its reciprocal constant decides."""
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


def values(wq, sg, zp, K, group):
    """w4_plain.values on the device."""
    byte, shift = (torch.from_numpy(a).to(DEV) for a in P.place(K))
    at = torch.arange(K, device=DEV) // group
    zero = 8.0 if zp is None else zp.T[:, at].double()
    return (((wq[:, byte] >> shift.to(torch.uint8)) & 15).double() - zero) * sg.T[:, at].double()


def random_weight(seed, N, K, group, asym):
    """Random bytes are codes where K is whole blocks; elsewhere the padding's nibbles are cleared."""
    gen = torch.Generator(DEV).manual_seed(seed)
    wq = torch.randint(0, 256, (N, P.row_bytes(K)), generator=gen, device=DEV, dtype=torch.uint8)
    if K % 128:
        keep = torch.from_numpy(P.pack(np.full((1, K), 15, np.uint8))).to(DEV)
        wq &= keep
    G = -(-K // group)
    sg = (0.01 * (0.5 + 1.5 * torch.rand(G, N, generator=gen, device=DEV))).to(torch.bfloat16)
    zp = torch.randint(0, 16, (G, N), generator=gen, device=DEV, dtype=torch.uint8) if asym else None
    return wq, sg, zp


# ------------------------------------------------------------------------------------------------ binary32 inputs
def whole_numbers_of_24_bits(rng, n):
    """Binary32 numbers whose last significand bit is set, so that each of their three bf16 parts is needed."""
    v = rng.integers(2 ** 23, 2 ** 24, n) | 1
    return (v * 2.0 ** rng.integers(-40, -6, n) * rng.choice([-1.0, 1.0], n)).astype(np.float32)


@pytest.mark.parametrize("M", [1, 2, 3, 4, 8, 9, 16, 17, 33, 70])
@pytest.mark.parametrize("N,K,group", [(40, 400, 32), (1001, 1040, 64), (2056, 2064, 128), (2056, 2064, 64),
                                       (4104, 4112, 32), (30008, 144, 128)])
def test_binary32_inputs_enter_whole(M, N, K, group):
    """One input a token, weights 0 or a power of two: each output is one product, which binary32 holds exactly, and
    every sum of parts on the way to it as well.  (From 9 tokens, sizes on either side of the batch kernel's rule.)"""
    rng = np.random.default_rng(M + N + K + group)
    codes = np.array([8, 9, 10, 12, 0, 7, 6, 4], np.uint8)[rng.integers(0, 8, (N, K))]  # 0, 1, 2, 4, -8, -1, -2, -4
    sg = (2.0 ** rng.integers(-3, 4, (-(-K // group), N))).astype(np.float32)
    wq = P.pack(codes)
    x = np.zeros((M, K), np.float32)
    at = rng.integers(0, K, M)
    at[0] = K - 1
    x[np.arange(M), at] = whole_numbers_of_24_bits(rng, M)
    want = x[np.arange(M), at][:, None].astype(np.float64) * P.values(wq, sg, None, K, group)[:, at].T
    assert np.array_equal(want.astype(np.float32), want)
    y = sq.sq_w4_gemm(dev(x), dev(wq), dev(sg, "bf16"), group=group, out_dtype=torch.float32)
    assert np.array_equal(y.double().cpu().numpy(), want)


# ------------------------------------------------------------------------------------------------ passes and chunks
@pytest.mark.parametrize("M,N,K,group,asym,dt", [
    (16, 40008, 3968, 128, False, "bf16"),   # a block has more tiles than cells beside x: passes of tiles, x kept
    (15, 53001, 4096, 64, False, "bf16"),    # the same, scales in single pieces
    (16, 1000, 49152, 128, False, "bf16"),   # x does not fit eight blocks: chunks of K
    (16, 10440, 49152, 128, True, "bf16"),   # chunks of K, and passes of tiles within
    (33, 2056, 49152, 64, False, "bf16"),    # three blocks of 16 tokens in chunks, beyond the batch kernel's reach
    (64, 1000, 49168, 32, True, "bf16"),     # a last unit of one block with one group in it
    (6, 20001, 12304, 128, True, "f32"),     # binary32 in chunks
])
def test_long_rows_and_many_tiles(M, N, K, group, asym, dt):
    wq, sg, zp = random_weight(M + N, N, K, group, asym)
    gen = torch.Generator(DEV).manual_seed(K)
    x = torch.randn(M, K, generator=gen, device=DEV)
    x[:, torch.randint(0, K, (K // 100,), generator=gen, device=DEV)] *= 50
    x = x.to(TD[dt])
    w = values(wq, sg, zp, K, group)
    ref = x.double() @ w.T
    bound = P.depth(K, group) * P.U * 1.01 * (x.double().abs() @ w.abs().T)
    del w
    y = sq.sq_w4_gemm(x, wq, sg, zp, group=group, out_dtype=torch.float32)
    assert ((y.double() - ref).abs() <= bound * (1 + 2.0 ** -24) + ref.abs() * P.HALF_STEP["f32"]).all()
    again = torch.full((M + 1, N + 3), -7.0, device=DEV)
    sq.sq_w4_gemm(x, wq, sg, zp, group=group, y=again[:M, 1:N + 1])
    assert torch.equal(again[:M, 1:N + 1], y)
    again[:M, 1:N + 1] = -7
    assert (again == -7).all()


# ------------------------------------------------------------------------------------------------ the quantiser's scale
@pytest.mark.parametrize("asym,parts", [(False, 7), (True, 15)])
def test_scale_beside_a_tie(asym, parts):
    """The ranges whose product with the rounded reciprocal and whose quotient round to different bf16 numbers: they lie
    beside the middle of two of them.  The scale is the product's, and no further from the quotient than half a step and
    2^-23 of it."""
    f = np.float32
    span = (np.arange(2 ** 23, 2 ** 24).astype(f) * f(2.0 ** -26))
    recip = P.bf16(span * (f(1) / f(parts)))
    odd = recip != P.bf16(span / f(parts))
    assert 0 < odd.sum() < 1000
    span = span[odd]
    span = span[:len(span) // 8 * 8]
    N = len(span)
    rng = np.random.default_rng(parts)
    W = (rng.uniform(0, 1, (32, N)) * span).astype(f)      # from 0 to the range, which row 5 has whole
    W[5] = span
    if not asym:
        W[::2] *= -1
    wq, sg, zp, _, _ = sq.sq_fold_quant_weights_w4(dev(W), group=32, asym=asym)
    codes, r_sg, r_zp = P.quantise(W, None, 32, asym)
    got = sg.float().cpu().numpy()[0]
    assert np.array_equal(got, recip[odd][:N]) and np.array_equal(got, r_sg[0])
    assert np.array_equal(wq.cpu().numpy(), P.pack(codes))
    assert not asym or np.array_equal(zp.cpu().numpy(), r_zp)
    exact = span.astype(np.float64) / parts
    half_step = 2.0 ** (np.floor(np.log2(exact)) - 8)
    assert (np.abs(got - exact) <= half_step + exact * 2.0 ** -23).all()
