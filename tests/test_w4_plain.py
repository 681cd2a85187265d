"""CPU: the packed 4-bit format, its plain quantiser, and the host-side checks of the library's 4-bit
entry points (every call below returns before any CUDA call is made)."""
import ctypes

import numpy as np
import pytest
import torch

import w4_plain as P
import w8a8_smoothquant_gemm_b200 as sq

INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 1, 2, 3, 5
F32, BF16, I32 = 0, 1, 2
A, B, C, D = (ctypes.c_void_p(0x10000 * i) for i in range(1, 5))
A8, A2 = ctypes.c_void_p(0x10008), ctypes.c_void_p(0x10002)
ODD = ctypes.c_void_p(0x10001)


@pytest.mark.parametrize("K", [16, 112, 128, 144, 1040])
def test_pack_round_trip(K):
    codes = np.random.default_rng(K).integers(0, 16, (5, K)).astype(np.uint8)
    wq = P.pack(codes)
    assert wq.shape == (5, sq.sq_w4_row_bytes(K)) == (5, P.row_bytes(K))
    assert np.array_equal(P.unpack(wq, K), codes)
    # every nibble of the padding is zero
    assert int(np.unpackbits(wq).sum()) == int(np.unpackbits(codes).sum())


def test_each_block_word_holds_eight_consecutive_codes():
    codes = (np.arange(128) % 16).astype(np.uint8)[None]
    word = P.pack(codes).view("<u4")[0]
    assert word[0] == 0x75316420       # k = 0 .. 7: even codes in the low half, odd ones in the high half
    assert word[4] == 0xFDB9ECA8       # byte 16 = lane 1: k = 8 .. 15
    assert word[1] == word[0]          # byte 4: k = 32 .. 39


@pytest.mark.parametrize("asym", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_plain_quantiser_is_nearest_on_its_grid(group, asym):
    rng = np.random.default_rng(group)
    W = rng.normal(0, 0.02, (208, 24)).astype(np.float32)
    s = rng.uniform(0.5, 2, 208).astype(np.float32)
    W[64:128, 3] = 0
    codes, sg, zp = P.quantise(W, s, group, asym)
    v = P.values(P.pack(codes), sg, zp, 208, group)
    step = sg[np.arange(208) // group].T
    # half a step, up to the clip at the ends: the bf16 scale may fall short by 2^-8 of 15 (7) steps
    assert (np.abs(v - (s[:, None] * W).T) <= step * (0.5 + 16 * 2.0 ** -8) + 1e-12).all()
    assert (v[3, 64:128] == 0).all()


def test_row_bytes():
    L = sq.lib()
    for K in (0, 16, 128, 144, 4096):
        assert L.sq_w4_row_bytes(K) == P.row_bytes(K) == sq.sq_w4_row_bytes(K)
    assert L.sq_w4_row_bytes(-1) == -1


def test_fold_refusals():
    def call(W=A, dt=BF16, K=256, N=64, ldw=64, s=B, gamma=None, beta=None, group=128, wq=C, sg=D, zp=None, gf=None,
             bf=None):
        return sq.lib().sq_fold_quant_weights_w4(W, dt, K, N, ldw, s, gamma, beta, group, wq, sg, zp, gf, bf, None)

    assert call(dt=I32) == INVALID and call(K=-16) == INVALID and call(N=-8) == INVALID
    assert call(W=None) == INVALID and call(wq=None) == INVALID and call(sg=None) == INVALID
    assert call(ldw=32) == INVALID and call(group=0) == INVALID and call(group=-32) == INVALID
    assert call(group=48) == UNSUPPORTED and call(group=256) == UNSUPPORTED
    assert call(W=A8) == ALIGN and call(wq=A8) == ALIGN and call(sg=ODD) == ALIGN
    assert call(N=60, ldw=64) == ALIGN and call(K=24) == ALIGN
    assert call(K=133152) == UNSUPPORTED
    assert call(s=A2) == INVALID
    assert call(K=0) == 0 and call(N=0) == 0


def test_dequant_refusals():
    def call(wq=A, sg=B, zp=None, K=256, N=64, group=128, y=C, ydt=BF16, ldy=256):
        return sq.lib().sq_w4_dequant(wq, sg, zp, K, N, group, y, ydt, ldy, None)

    assert call(K=-1) == INVALID and call(N=-1) == INVALID and call(ydt=I32) == INVALID
    assert call(wq=None) == INVALID and call(sg=None) == INVALID and call(y=None) == INVALID
    assert call(ldy=128) == INVALID and call(group=0) == INVALID and call(group=16) == UNSUPPORTED
    assert call(y=A8) == ALIGN and call(ldy=260) == ALIGN and call(K=24, ldy=256) == ALIGN
    assert call(K=133152, ldy=133152) == UNSUPPORTED
    assert call(K=0) == 0 and call(N=0) == 0


def test_gemm_refusals():
    def call(x=A, dt=BF16, M=4, K=256, ldx=256, wq=B, sg=C, zp=None, N=64, group=128, y=D, ydt=BF16, ldy=64):
        return sq.lib().sq_w4_gemm(x, dt, M, K, ldx, wq, sg, zp, N, group, y, ydt, ldy, None)

    assert call(M=-1) == INVALID and call(N=-1) == INVALID and call(K=0) == INVALID
    assert call(dt=I32) == INVALID and call(ydt=I32) == INVALID
    assert call(x=None) == INVALID and call(wq=None) == INVALID and call(sg=None) == INVALID and call(y=None) == INVALID
    assert call(ldx=128) == INVALID and call(ldy=32) == INVALID
    assert call(group=0) == INVALID and call(group=96) == UNSUPPORTED
    assert call(x=A8) == ALIGN and call(ldx=260) == ALIGN and call(wq=A8) == ALIGN and call(y=ODD) == ALIGN
    assert call(K=24, ldx=24) == ALIGN
    assert call(K=133152, ldx=133152) == UNSUPPORTED and call(M=65537) == UNSUPPORTED
    assert call(M=0) == 0 and call(N=0) == 0


def moe(**kw):
    a = dict(x=A, dt=BF16, T=4, D=256, ldx=256, wr=B, rdt=BF16, E=8, k=2, renorm=1, ids=A, wts=B, w13=C, s13=D, z13=None,
             w2=C, s2=D, z2=None, F=128, group=128, y=A, ydt=BF16, ldy=256, ws=B, bytes=1 << 30)
    assert set(kw) <= set(a)
    return sq.lib().sq_moe_w4(*{**a, **kw}.values(), None)


def test_moe_refusals():
    for bad in (dict(T=-1), dict(D=0), dict(F=0), dict(E=0), dict(k=0), dict(k=9), dict(renorm=2), dict(dt=I32),
                dict(rdt=I32), dict(ydt=I32), dict(x=None), dict(wr=None), dict(ids=None), dict(wts=None),
                dict(w13=None), dict(s13=None), dict(w2=None), dict(s2=None), dict(y=None), dict(z13=A), dict(z2=A),
                dict(ldx=128), dict(ldy=128), dict(group=0)):
        assert moe(**bad) == INVALID, bad
    for bad in (dict(x=A8), dict(ldx=260), dict(wr=A8), dict(w13=A8), dict(w2=A8), dict(y=ODD), dict(ids=A2),
                dict(wts=A2), dict(s13=ODD), dict(s13=A8), dict(s2=A8), dict(z13=A8, z2=A), dict(F=120), dict(D=248, ldx=248), dict(ws=A8)):
        assert moe(**bad) == ALIGN, bad
    for bad in (dict(T=65), dict(E=1025), dict(E=64, k=33), dict(group=16), dict(F=133152), dict(D=131072, ldx=131072, ldy=131072, F=131072)):
        assert moe(**bad) == UNSUPPORTED, bad
    size = sq.sq_moe_w4_workspace_size(4, 256, 128, 8, 2)
    assert moe(ws=None) == WORKSPACE and moe(bytes=size - 1) == WORKSPACE
    assert moe(T=0) == 0


def test_moe_routed_refusals():
    def call(**kw):
        a = dict(x=A, dt=BF16, T=4, D=256, ldx=256, ids=A, wts=B, E=8, k=2, w13=C, s13=D, z13=None, w2=C, s2=D, z2=None,
                 F=128, group=128, y=A, ydt=BF16, ldy=256, ws=B, bytes=1 << 30)
        return sq.lib().sq_moe_w4_routed(*{**a, **kw}.values(), None)

    assert call(ids=None) == INVALID and call(wts=None) == INVALID and call(k=0) == INVALID
    assert call(ids=A2) == ALIGN and call(T=65) == UNSUPPORTED and call(ws=None) == WORKSPACE
    assert call(T=0) == 0


def test_moe_workspace_size():
    size = sq.lib().sq_moe_w4_workspace_size
    assert size(1, 256, 128, 8, 2) > 0
    assert size(8, 256, 128, 8, 2) >= size(1, 256, 128, 8, 2)
    for bad in ((65, 256, 128, 8, 2), (1, 0, 128, 8, 2), (1, 256, 128, 8, 9), (1, 256, 128, 1025, 2)):
        assert size(*bad) == 2 ** 64 - 1
        with pytest.raises(ValueError):
            sq.sq_moe_w4_workspace_size(*bad)


def test_moe_workspace_serves_smaller_sizes():
    """The size grows with every argument, also where the experts' lists change their shape."""
    size = sq.sq_moe_w4_workspace_size
    for E in (1, 2, 5, 8, 15, 33, 128):
        for k in (1, 2, 5, 8, 15, 32):
            if k > E:
                continue
            of_T = [size(T, 16, 16, E, k) for T in range(1, 65)]
            assert of_T == sorted(of_T)
            for T in (1, 7, 8, 9, 16, 33, 64):
                assert size(T, 16, 16, E, k) <= size(T, 16, 16, E + 1, k)
                assert k in (E, 32) or size(T, 16, 16, E, k) <= size(T, 16, 16, E, k + 1)


def test_binding_refuses_what_the_call_could_not_see():
    """Shapes, types and devices: checked before a pointer is taken."""
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    wq, sg = torch.zeros(8, 128, dtype=torch.uint8), torch.zeros(2, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sq.sq_w4_gemm(x, wq, sg)                                   # host tensors
    with pytest.raises(ValueError):
        sq.sq_w4_dequant(wq, sg, K=256)                            # host tensors
    with pytest.raises(ValueError):
        sq.sq_w4_dequant(wq, sg, K=512)                            # rows of another K
    with pytest.raises(ValueError):
        sq.sq_w4_dequant(wq, sg.float(), K=256)                    # scales of another type
    with pytest.raises(ValueError):
        sq.sq_w4_dequant(wq, sg, torch.zeros(2, 8), K=256)         # zero points of another type
    with pytest.raises(ValueError):
        sq.sq_w4_dequant(wq, sg, K=256, group=48)
    with pytest.raises(ValueError):
        sq.sq_fold_quant_weights_w4(torch.zeros(256, 8, dtype=torch.bfloat16))


def test_binding_refuses_a_stream_of_another_device():
    import types
    there = types.SimpleNamespace(device_index=0)
    x = torch.zeros(2, 256, dtype=torch.bfloat16)  # not on device 0
    wq, sg = torch.zeros(8, 128, dtype=torch.uint8), torch.zeros(2, 8, dtype=torch.bfloat16)
    w13, s13 = torch.zeros(2, 32, 128, dtype=torch.uint8), torch.zeros(2, 2, 32, dtype=torch.bfloat16)
    ids, wts = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1)
    for call in (lambda: sq.sq_w4_gemm(x, wq, sg, stream=there), lambda: sq.sq_w4_dequant(wq, sg, K=256, stream=there),
                 lambda: sq.sq_fold_quant_weights_w4(x, stream=there),
                 lambda: sq.sq_moe_w4(x, x, 1, w13, s13, w13, s13, stream=there),
                 lambda: sq.sq_moe_w4_routed(x, ids, wts, w13, s13, w13, s13, stream=there)):
        with pytest.raises(ValueError, match="another device"):
            call()
