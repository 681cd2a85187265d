"""4-bit operators at the ends of their ranges, in one graph, and beside the INT8 kernels."""
import numpy as np
import pytest
import torch

import w4_plain as P
import w8a8_smoothquant_gemm_b200 as sq
from test_gpu_moe import W_OFF, Layer, check, dev, num
from test_gpu_w4 import activations, random_weight

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
MAX_K = 133136


@pytest.mark.parametrize("asym", [False, True])
def test_fold_and_values_of_the_longest_rows(asym):
    rng = np.random.default_rng(1)
    W = P.bf16(rng.normal(0, 0.02, (MAX_K, 8)).astype(np.float32))
    s = rng.uniform(0.2, 3, MAX_K).astype(np.float32)
    wq, sg, zp, _, _ = sq.sq_fold_quant_weights_w4(dev(W, "bf16"), dev(s), group=64, asym=asym)
    codes, r_sg, r_zp = P.quantise(W, s, 64, asym)
    assert np.array_equal(sg.float().cpu().numpy(), r_sg) and np.array_equal(wq.cpu().numpy(), P.pack(codes))
    assert not asym or np.array_equal(zp.cpu().numpy(), r_zp)
    v = sq.sq_w4_dequant(wq, sg, zp, K=MAX_K, group=64, out_dtype=torch.float32)
    assert np.array_equal(num(v), P.values(P.pack(codes), r_sg, r_zp, MAX_K, 64))


def test_values_of_more_rows_than_a_grid_has():
    K, N = 16, 1_100_003
    codes = torch.randint(0, 16, (N, K), device=DEV, dtype=torch.uint8)
    byte, shift = P.place(K)
    wq = torch.zeros(N, 64, dtype=torch.uint8, device=DEV)
    for k in range(K):
        wq[:, byte[k]] |= codes[:, k] << int(shift[k])
    sg = (torch.rand(1, N, device=DEV) + 0.5).to(torch.bfloat16)
    zp = torch.randint(0, 16, (1, N), device=DEV, dtype=torch.uint8)
    v = sq.sq_w4_dequant(wq, sg, zp, K=K, group=32, out_dtype=torch.float32)
    assert torch.equal(v, (codes.float() - zp.T.float()) * sg.T.float())


@pytest.mark.parametrize("K,N,dt", [(16, 8, "bf16"), (144, 17, "f32"), (4096, 1032, "bf16"), (2064, 2056, "f32")])
def test_product_of_the_most_tokens(K, N, dt):
    """65536 tokens, either kernel; the rows of a sample against 64 bits, and the rows behind."""
    M, group = 65536, 64
    rng = np.random.default_rng(K)
    (wq, sg, zp), w = random_weight(rng, K, N, group, True)
    x = torch.randn(M, K, generator=torch.Generator(DEV).manual_seed(K), device=DEV)
    x = x.to(torch.bfloat16) if dt == "bf16" else x
    y = torch.full((M + 1, N), -7.0, device=DEV)
    sq.sq_w4_gemm(x, wq, sg, zp, group=group, y=y[:M])
    rows = torch.cat([torch.arange(0, M, 1021), torch.tensor([1, 63, 64, M - 65, M - 2, M - 1])]).to(DEV)
    check(y[rows], *P.product(num(x[rows]), w, group), "f32")
    assert (y[M] == -7).all()
    with pytest.raises(sq.SQError):
        sq.sq_w4_gemm(torch.zeros(M + 1, 16, dtype=torch.bfloat16, device=DEV), *random_weight(rng, 16, 8, 32, False)[0][:2], group=32)


@pytest.mark.parametrize("T,E,k,D,F,dt", [(64, 1024, 32, 16, 16, "bf16"), (64, 2, 1, MAX_K, 16, "bf16"), (1, 2, 2, MAX_K, 16, "f32"),
                                          (9, 2, 2, 16, MAX_K, "bf16"), (1, 3, 1, 16, MAX_K, "f32")])
def test_layer_at_its_limits(T, E, k, D, F, dt):
    L = Layer(T + E, E, D, F, 128, True, dt)
    x = L.x(T)
    y, ids, wts = sq.sq_moe_w4(dev(x, dt), dev(L.wr, dt), k, *L.weights(), **L.kw(), out_dtype=torch.float32)
    r_ids, r_w = P.choose(x, L.wr, k, True)
    assert np.array_equal(ids.cpu().numpy(), r_ids)
    check(y, *L.ref(x, r_ids, r_w, W_OFF), "f32")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("ids", [[2, -1, 6, 2], [3, 3, 3, 3], [-1, -1, -1, -1], [5, 0, 1 << 30, -5], [4] * 3 + [1]])
def test_one_token_with_masked_and_repeated_choices(ids, dt):
    L = Layer(21, 6, 144, 80, 32, True, dt)
    x, ids = L.x(1), np.array([ids], np.int32)
    wts = L.rng.uniform(-1, 1, ids.shape).astype(np.float32)
    used = np.where((ids >= 0) & (ids < 6), ids, -1)
    wts[used < 0] = np.nan  # not looked at
    y = sq.sq_moe_w4_routed(dev(x, dt), dev(ids), dev(wts), *L.weights(), **L.kw(), out_dtype=torch.float32)
    check(y, *L.ref(x, used, np.where(used < 0, 0, wts)), "f32")
    assert (used >= 0).any() or (y == 0).all()


def test_masked_choices_of_many_tokens_are_not_looked_at():
    L = Layer(22, 6, 144, 80, 32, False, "bf16")
    x = L.x(12)
    ids = L.rng.integers(0, 6, (12, 5)).astype(np.int32)
    wts = L.rng.uniform(-1, 1, ids.shape).astype(np.float32)
    gone = L.rng.random(ids.shape) < 0.5
    ids[gone], wts[gone] = L.rng.choice([-1, 6, -(1 << 31), (1 << 31) - 1], int(gone.sum())), np.nan
    y = sq.sq_moe_w4_routed(dev(x, "bf16"), dev(ids), dev(wts), *L.weights(), **L.kw(), out_dtype=torch.float32)
    check(y, *L.ref(x, np.where(gone, -1, ids), np.where(gone, 0, wts)), "f32")


@pytest.mark.parametrize("T", [1, 11])
def test_binary32_tokens_with_a_bf16_router(T):
    L = Layer(23, 12, 272, 48, 64, False, "f32")
    x, wr = L.x(T), P.bf16(L.wr)
    _, ids, wts = sq.sq_moe_w4(dev(x), dev(wr, "bf16"), 3, *L.weights(), **L.kw())
    r_ids, r_w = P.choose(x, wr, 3, True)
    assert np.array_equal(ids.cpu().numpy(), r_ids) and (np.abs(num(wts) - r_w) <= r_w * W_OFF).all()


def test_fold_values_product_and_layer_in_one_graph():
    """Weights quantised, read back, multiplied and used as experts within one capture, replayed with other weights."""
    K, N, group = 512, 1040, 64
    gen = torch.Generator(DEV).manual_seed(3)
    W = torch.empty(K, 2 * K, device=DEV)
    down = torch.empty(K, K, device=DEV)
    x = torch.empty(20, K, device=DEV)
    wr = torch.randn(4, K, generator=gen, device=DEV)
    ws = sq.sq_moe_w4_workspace(20, K, K, 1, 1)

    def call():
        wq, sg, zp, _, _ = sq.sq_fold_quant_weights_w4(W, group=group, asym=True)
        dq, ds, dz, _, _ = sq.sq_fold_quant_weights_w4(down, group=group, asym=True)
        v = sq.sq_w4_dequant(wq, sg, zp, K=K, group=group, out_dtype=torch.float32)
        y = sq.sq_w4_gemm(x, wq, sg, zp, group=group, out_dtype=torch.float32)
        z, ids, wts = sq.sq_moe_w4(x, wr[:1].contiguous(), 1, wq[None], sg[None], dq[None], ds[None], z13=zp[None],
                                   z2=dz[None], group=group, out_dtype=torch.float32, workspace=ws)
        return wq, sg, zp, v, dq, ds, dz, y, z, ids, wts

    def fill(seed):
        g = torch.Generator(DEV).manual_seed(seed)
        for t, by in ((W, 0.03), (down, 0.03), (x, 1.0)):
            t.copy_(torch.randn(t.shape, generator=g, device=DEV) * by)

    fill(0)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    for seed in (1, 2):
        fill(seed)
        want = call()
        torch.cuda.synchronize()
        for t in held:
            t.zero_()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))
        check(want[7], *P.product(num(x), num(want[3]), group), "f32")


def test_beside_the_int8_kernels():
    """4-bit products of either kernel and layers between INT8 quantisers and GEMMs, back to back and on two streams: each
    gives what it gives alone (programmatic launches and tensor memory of one must not touch the other's)."""
    rng = np.random.default_rng(31)
    K, N = 2048, 2304
    (wq, sg, zp), w = random_weight(rng, K, N, 128, True)
    x = [dev(activations(rng, m, K, "bf16"), "bf16") for m in (3, 64)]
    W = dev(P.bf16(rng.normal(0, 0.03, (K, N)).astype(np.float32)), "bf16")
    s = torch.ones(K, device=DEV)
    w8, sw, _, _ = sq.sq_fold_quant_weights(W, s)
    L = Layer(32, 8, K, 256, 128, False, "bf16")
    wr = dev(L.wr, "bf16")
    rows = dev(activations(rng, 512, K, "bf16"), "bf16")

    def chain(workspace):
        out = []
        for a in (x[0], x[1], rows):
            xq, sx = sq.sq_ln_smooth_quant(a, s=s)
            out.append(sq.sq_w4_gemm(x[1], wq, sg, zp))
            out.append(sq.sq_w8a8_gemm(xq, sx, w8, sw))
            out.append(sq.sq_w4_gemm(x[0], wq, sg, zp))
            h = out[-2][:64, :K]
            xq, sx = sq.sq_ln_smooth_quant(h, s=s)
            out.append(sq.sq_w8a8_gemm(xq, sx, w8, sw))
            out.append(sq.sq_w4_gemm(out[-1][:, :K], wq, sg, zp))
            out += sq.sq_moe_w4(x[1], wr, 2, *L.weights(), **L.kw(), workspace=workspace)
        return out

    spaces = [sq.sq_moe_w4_workspace(64, K, 256, 8, 2) for _ in range(2)]
    want = chain(spaces[0])
    check(want[0], *P.product(num(x[1]), w, 128), "bf16")
    check(want[4], *P.product(num(want[3][:, :K]), w, 128), "bf16")
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for st, ws in zip(streams, spaces):
            with torch.cuda.stream(st):
                got.append(chain(ws))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for run in got for a, b in zip(run, want))
    assert sq.sq_device_error() == 0
