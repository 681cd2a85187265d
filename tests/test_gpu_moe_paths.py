"""The mixture-of-experts layer on the ways that large batches take: tokens read from global memory, several passes of
tiles in either kernel; and the bits of x and of h that enter the products."""
import numpy as np
import pytest
import torch

import w4_plain as P
import w8a8_smoothquant_gemm_b200 as sq
from test_gpu_moe import W_OFF, Layer, check, dev

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# The expert kernels' shared memory, restated from their launch: which sizes take which way.
BUDGET, WARPS = 226 * 1024, 16


def up16(n):
    return -(-n // 16) * 16


def plan(T, D, F, E, k, group, asym, dt):
    """(x staged, gate/up passes' tiles, tiles of a block at most, h staged, down passes' tiles, tiles of a block)."""
    sms = torch.cuda.get_device_properties(DEV).multi_processor_count
    S, SH = (1, 2) if dt == "bf16" else (3, 3)
    entry = 8 if T <= 8 or T * k <= 4 * E else 16
    entries, slots = min(T * k, E + T * k // entry), T * k
    per_unit = 2 * (4 // (group // 32))
    ring = WARPS * 2 * (2048 + per_unit * 32 + (per_unit * 16 if asym else 0))
    lists = up16((2 + 2 * entries + 2 * slots) * 4)
    rings = max(ring, up16(12 * E + 8 * slots))

    def pitch(K):
        return -(-K // 256) * 512 + 64

    def fit(room, cell, tiles):
        return min(tiles, room // cell - (WARPS - 1))

    per = -(-min(E, T * k) * (F // 8) // sms)
    cell, x = 128 * (entry // 8) * 4, S * T * pitch(D)
    x_staged = fit(BUDGET - lists - rings - x, cell, per) >= min(per, 16)
    up = fit(BUDGET - rings - lists - (x if x_staged else 0), cell, per)
    tiles, cell2, C = -(-D // 16), T * 80, 1
    while C < 8 and tiles * C * 2 <= sms:
        C *= 2
    h = SH * slots * pitch(F)
    h_staged = fit(BUDGET - lists - ring - h, cell2, 2) >= 2
    per2 = -(-tiles // min(tiles, sms // C))
    down = min(fit(BUDGET - lists - (h if h_staged else 0) - ring, cell2, per2), max(1, ring // (T * 64)))
    return x_staged, up, lambda active: -(-active * (F // 8) // sms), h_staged, down, per2


@pytest.mark.parametrize("T,E,k,D,F,group,asym,dt", [(32, 8, 2, 4096, 208, 128, False, "bf16"),
                                                     (64, 16, 4, 2064, 144, 64, True, "bf16"),
                                                     (40, 5, 2, 4112, 80, 32, True, "bf16"),
                                                     (32, 8, 2, 2048, 256, 128, False, "f32"),
                                                     (64, 6, 3, 1040, 144, 32, True, "f32")])
def test_tokens_from_global_memory(T, E, k, D, F, group, asym, dt):
    """x of many tokens does not fit shared memory: the gate/up kernel reads it where it lies, binary32 x as the parts that
    a kernel of its own has made."""
    assert not plan(T, D, F, E, k, group, asym, dt)[0]
    L = Layer(T + D, E, D, F, group, asym, dt)
    x = L.x(T)
    wide = torch.full((T + 1, D + 32), float("nan"), device=DEV, dtype=dev(x, dt).dtype)
    wide[:T, 16:D + 16] = dev(x, dt)
    xd, wr = wide[:T, 16:D + 16], dev(L.wr, dt)
    r_ids, r_w = P.choose(x, L.wr, k, True)
    y, ids, wts = sq.sq_moe_w4(xd, wr, k, *L.weights(), **L.kw(), out_dtype=torch.float32)
    assert np.array_equal(ids.cpu().numpy(), r_ids)
    assert (np.abs(wts.double().cpu().numpy() - r_w) <= r_w * W_OFF).all()
    check(y, *L.ref(x, r_ids, r_w, W_OFF), "f32")
    again = sq.sq_moe_w4_routed(dev(x, dt), ids, wts, *L.weights(), **L.kw(), out_dtype=torch.float32)
    assert torch.equal(y, again)
    # fewer tokens are staged, and give the same choices
    few = sq.sq_moe_w4(xd[:2], wr, k, *L.weights(), **L.kw(), out_dtype=torch.float32)
    assert plan(2, D, F, E, k, group, asym, dt)[0] and torch.equal(few[1], ids[:2])
    check(few[0], *L.ref(x[:2], r_ids[:2], r_w[:2], W_OFF), "f32")


@pytest.mark.parametrize("dt,T,D,staged", [("bf16", 64, 144, True), ("bf16", 64, 4096, False), ("f32", 64, 1040, False)])
def test_gate_and_up_in_several_passes(dt, T, D, staged):
    """All tokens on one of two experts: more entries than the passes were laid out for."""
    E, F, group = 2, 1200, 64
    x_staged, up, tiles, *_ = plan(T, D, F, E, 1, group, True, dt)
    assert x_staged == staged and tiles(T // 16) > up
    L = Layer(D, E, D, F, group, True, dt)
    x = L.x(T)
    ids, wts = np.ones((T, 1), np.int32), np.linspace(-2, 2, T, dtype=np.float32)[:, None]
    y = sq.sq_moe_w4_routed(dev(x, dt), dev(ids), dev(wts), *L.weights(), **L.kw(), out_dtype=torch.float32)
    check(y, *L.ref(x, ids, wts), "f32")


@pytest.mark.parametrize("T,D,F,staged", [(56, 16592, 16, True), (64, 14400, 32, True), (64, 37904, 272, False)])
def test_down_in_several_passes(T, D, F, staged):
    E, group = 3, 128
    *_, h_staged, down, per = plan(T, D, F, E, 1, group, False, "bf16")
    assert h_staged == staged and down < per
    L = Layer(D, E, D, F, group, False, "bf16")
    x = L.x(T)
    ids = L.rng.integers(-1, E, (T, 1)).astype(np.int32)
    wts = L.rng.uniform(-1, 1, (T, 1)).astype(np.float32)
    y = sq.sq_moe_w4_routed(dev(x, "bf16"), dev(ids), dev(wts), *L.weights(), **L.kw(), out_dtype=torch.float32)
    check(y, *L.ref(x, ids, wts), "f32")


@pytest.mark.parametrize("T", [1, 2, 3, 4, 9, 24, 64])
@pytest.mark.parametrize("D,F,dt", [(144, 80, "f32"), (1040, 272, "f32"), (144, 80, "bf16"), (4112, 272, "bf16")])
def test_the_bits_of_x_and_h_that_enter(T, D, F, dt):
    """Each row of a gate has its weights on the first half of the channels and each row of an up on the second, a token
    has one input in each half, and a row of W2 has one weight, all of them powers of two: an h is one product, an output
    is one h.  The gate is above 32, where silu(v) = v in binary32.  For a binary32 layer the up's input has 24 bits and
    the gate's is a power of two; for bf16 both have 8, and h the 16 of their product.  All of it has to come out."""
    rng = np.random.default_rng(T + D)
    E, group, half = 4, 32, D // 2
    powers = np.array([9, 10, 12], np.uint8)  # 1, 2, 4

    def weight(N, K, there):
        codes = np.where(there, powers[rng.integers(0, 3, (N, K))], np.uint8(8))
        return P.pack(codes), (2.0 ** rng.integers(-2, 3, (-(-K // group), N))).astype(np.float32), codes

    up, down, values13, values2 = [], [], [], []
    for _ in range(E):
        there = np.zeros((2 * F, D), bool)
        there[:F, :half], there[F:, half:] = True, True
        wq, sg, _ = weight(2 * F, D, there)
        up.append((wq, sg))
        values13.append(P.values(wq, sg, None, D, group))
        there = np.zeros((D, F), bool)
        there[np.arange(D), rng.integers(0, F, D)] = True
        wq, sg, _ = weight(D, F, there)
        down.append((wq, sg))
        values2.append(P.values(wq, sg, None, F, group))
    x = np.zeros((T, D), np.float32)
    first, second = rng.integers(0, half, T), rng.integers(half, D, T)
    second[0] = D - 1
    if dt == "f32":
        x[np.arange(T), first] = 2.0 ** rng.integers(7, 12, T)
        x[np.arange(T), second] = (rng.integers(2 ** 23, 2 ** 24, T) | 1) * 2.0 ** -20 * rng.choice([-1, 1], T)
    else:
        x[np.arange(T), first] = (rng.integers(2 ** 7, 2 ** 8, T) | 1) * 2.0
        x[np.arange(T), second] = (rng.integers(2 ** 7, 2 ** 8, T) | 1) * 2.0 ** -5 * rng.choice([-1, 1], T)
    ids = rng.integers(0, E, (T, 1)).astype(np.int32)
    wts = (2.0 ** rng.integers(-3, 4, (T, 1))).astype(np.float32)
    want = np.zeros((T, D))
    for t in range(T):
        gu = values13[ids[t, 0]] @ x[t].astype(np.float64)
        assert gu[:F].min() >= 32
        want[t] = wts[t, 0] * (values2[ids[t, 0]] @ (gu[:F] * gu[F:]))
    assert np.array_equal(want.astype(np.float32), want)
    stack = [dev(np.stack([p[i] for p in w]), "bf16" if i else None) for w in (up, down) for i in (0, 1)]
    y = sq.sq_moe_w4_routed(dev(x, dt), dev(ids), dev(wts), *stack, group=group, out_dtype=torch.float32)
    assert np.array_equal(y.double().cpu().numpy(), want)
