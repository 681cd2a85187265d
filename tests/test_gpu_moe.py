"""The mixture-of-experts layer with 4-bit experts against binary64 (w4_plain): routing, expert sums, masks, repeats."""
import numpy as np
import pytest
import torch

import w4_plain as P
import w8a8_smoothquant_gemm_b200 as sq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TD = {"bf16": torch.bfloat16, "f32": torch.float32}
H_PART = {"bf16": 2.0 ** -16, "f32": 2.0 ** -22}  # two rounded bf16 parts of h; three cut ones
# softmax weights: expf of a difference below 32 in magnitude rounded to binary32 (2^-24 * 32), its own error (2^-23),
# the sum's and the quotients' roundings
W_OFF = 2.0 ** -18


def dev(a, dt=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dt is None else t.to(TD[dt])


def num(t):
    return t.detach().double().cpu().numpy()


class Layer:
    def __init__(self, seed, E, D, F, group, asym, dt):
        rng = np.random.default_rng(seed)
        self.E, self.D, self.F, self.group, self.dt = E, D, F, group, dt

        def weight(K, N):
            codes = np.clip(np.rint(rng.normal(0, 2.6, (N, K))) + 8, 0, 15).astype(np.uint8)
            G = -(-K // group)
            sg = P.bf16(rng.uniform(0.5, 1.5, (G, N)).astype(np.float32) / np.float32(3 * np.sqrt(K)))
            zp = rng.integers(6, 11, (G, N)).astype(np.uint8) if asym else None
            return P.pack(codes), sg, zp

        up, down = [weight(D, 2 * F) for _ in range(E)], [weight(F, D) for _ in range(E)]
        self.host13, self.host2 = up, down

        def stack(parts, i, dtype=None):
            return None if parts[0][i] is None else dev(np.stack([p[i] for p in parts]), dtype)

        self.w13, self.s13, self.z13 = stack(up, 0), stack(up, 1, "bf16"), stack(up, 2)
        self.w2, self.s2, self.z2 = stack(down, 0), stack(down, 1, "bf16"), stack(down, 2)
        wr = rng.normal(0, 1.5 / np.sqrt(D), (E, D)).astype(np.float32)
        self.wr = P.bf16(wr) if dt == "bf16" else wr
        self.rng = rng

    def x(self, T):
        x = self.rng.normal(0, 1, (T, self.D)).astype(np.float32)
        return P.bf16(x) if self.dt == "bf16" else x

    def weights(self):
        return self.w13, self.s13, self.w2, self.s2

    def kw(self):
        return dict(z13=self.z13, z2=self.z2, group=self.group)

    def ref(self, x, ids, wts, w_off=0.0):
        def val(host, K):
            return lambda e: P.values(host[e][0], host[e][1], host[e][2], K, self.group)
        return P.experts(x, ids, wts, val(self.host13, self.D), val(self.host2, self.F), self.group, H_PART[self.dt],
                         w_off)


def check(y, ref, bound, out):
    off = np.abs(num(y) - ref)
    assert (off <= bound + np.abs(ref) * P.HALF_STEP[out] * (1 + 2.0 ** -8) + bound * P.HALF_STEP[out]).all(), (
        float((off - bound).max()))


@pytest.mark.parametrize("T", [1, 2, 5, 9, 17, 40, 64])
@pytest.mark.parametrize("E,k,D,F,group,asym,dt", [(8, 2, 256, 128, 128, False, "bf16"), (9, 3, 144, 208, 32, True, "f32"),
                                                   (4, 4, 272, 16, 64, True, "bf16"), (128, 8, 128, 48, 64, False, "bf16"),
                                                   (1, 1, 16, 16, 32, False, "f32")])
def test_layer(T, E, k, D, F, group, asym, dt):
    L = Layer(T + E, E, D, F, group, asym, dt)
    x = L.x(T)
    r_ids, r_w = P.choose(x, L.wr, k, True)
    ws = sq.sq_moe_w4_workspace(T, D, F, E, k)
    for out, renorm in (("bf16", True), ("f32", False)):
        y, ids, wts = sq.sq_moe_w4(dev(x, dt), dev(L.wr, dt), k, *L.weights(), **L.kw(), renorm=renorm, out_dtype=TD[out],
                                   workspace=ws)
        r_w = P.choose(x, L.wr, k, renorm)[1]
        assert np.array_equal(ids.cpu().numpy(), r_ids)
        assert (np.abs(num(wts) - r_w) <= r_w * W_OFF).all()
        check(y, *L.ref(x, r_ids, r_w, W_OFF), out)
    y2 = sq.sq_moe_w4_routed(dev(x, dt), ids, wts, *L.weights(), **L.kw(), out_dtype=torch.float32, workspace=ws)
    assert torch.equal(y, y2)  # the same experts and weights: the same sums


@pytest.mark.parametrize("T,E,k,D,F", [(1, 8, 2, 4096, 1024), (3, 16, 4, 1040, 720), (16, 8, 2, 2048, 1408)])
def test_layer_sizes(T, E, k, D, F):
    L = Layer(D, E, D, F, 128, False, "bf16")
    x = L.x(T)
    y, ids, wts = sq.sq_moe_w4(dev(x, "bf16"), dev(L.wr, "bf16"), k, *L.weights(), **L.kw(), out_dtype=torch.float32)
    r_ids, r_w = P.choose(x, L.wr, k, True)
    assert np.array_equal(ids.cpu().numpy(), r_ids)
    check(y, *L.ref(x, r_ids, r_w, W_OFF), "f32")


def test_equal_logits_go_to_the_lowest_index():
    L = Layer(1, 40, 64, 32, 32, False, "bf16")
    wr = np.repeat(L.wr[:8], 5, 0)  # each router row five times
    x = L.x(6)
    _, ids, wts = sq.sq_moe_w4(dev(x, "bf16"), dev(wr, "bf16"), 7, *L.weights(), **L.kw())
    r_ids, r_w = P.choose(x, wr, 7, True)
    assert np.array_equal(ids.cpu().numpy(), r_ids)
    zero = np.zeros_like(wr)
    _, ids, wts = sq.sq_moe_w4(dev(x, "bf16"), dev(zero, "bf16"), 7, *L.weights(), **L.kw(), renorm=False)
    assert (ids.cpu().numpy() == np.arange(7)).all()
    assert (np.abs(num(wts) - 1 / 40) <= W_OFF / 40).all()


def test_router_types_differ_from_the_layers():
    L = Layer(2, 8, 256, 64, 64, False, "bf16")
    x, wr32 = L.x(4), L.rng.normal(0, 0.1, (8, 256)).astype(np.float32)
    _, ids, wts = sq.sq_moe_w4(dev(x, "bf16"), dev(wr32), 3, *L.weights(), **L.kw())
    r_ids, r_w = P.choose(x, wr32, 3, True)
    assert np.array_equal(ids.cpu().numpy(), r_ids) and (np.abs(num(wts) - r_w) <= r_w * W_OFF).all()


def test_many_experts_and_choices():
    L = Layer(3, 1000, 32, 16, 32, False, "f32")
    x = L.x(64)
    y, ids, wts = sq.sq_moe_w4(dev(x), dev(L.wr), 32, *L.weights(), **L.kw(), out_dtype=torch.float32)
    r_ids, r_w = P.choose(x, L.wr, 32, True)
    assert np.array_equal(ids.cpu().numpy(), r_ids)
    check(y, *L.ref(x, r_ids, r_w, W_OFF), "f32")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_given_choices_masked_repeated_and_one_sided(dt):
    L = Layer(4, 6, 144, 80, 32, True, dt)
    T, k = 21, 4
    x = L.x(T)
    ids = L.rng.integers(0, 6, (T, k)).astype(np.int32)   # repeats among them
    wts = L.rng.uniform(-1, 1, (T, k)).astype(np.float32)
    ids[3] = -1                                            # a token with no expert
    ids[4] = [2, -1, 6, 1 << 30]                           # masked and out of range
    ids[5] = 3                                             # one expert, four times
    ids[6:] = np.where(ids[6:] == 0, 1, ids[6:])           # expert 0: hardly a token
    wts[7] = 0
    y = torch.full((T + 1, 150), -7.0, device=DEV)
    sq.sq_moe_w4_routed(dev(x, dt), dev(ids), dev(wts), *L.weights(), **L.kw(), y=y[:T, 3:147])
    used = np.where((ids >= 0) & (ids < 6), ids, -1)
    check(y[:T, 3:147], *L.ref(x, used, wts), "f32")
    assert (y[3, 3:147] == 0).all()
    y[:T, 3:147] = -7
    assert (y == -7).all()


def test_all_tokens_on_one_expert_and_none_at_all():
    L = Layer(5, 5, 256, 112, 64, False, "bf16")
    x = L.x(64)
    ids, wts = np.full((64, 1), 4, np.int32), np.ones((64, 1), np.float32)
    y = sq.sq_moe_w4_routed(dev(x, "bf16"), dev(ids), dev(wts), *L.weights(), **L.kw(), out_dtype=torch.float32)
    check(y, *L.ref(x, ids, wts), "f32")
    y = sq.sq_moe_w4_routed(dev(x, "bf16"), dev(ids * 0 - 1), dev(wts), *L.weights(), **L.kw())
    assert (y == 0).all()


def test_nan_stays_in_its_token():
    L = Layer(6, 8, 256, 64, 128, False, "bf16")
    x = L.x(9)
    bad = x.copy()
    bad[2, 5], bad[7, 0] = np.nan, np.inf
    y, ids, wts = sq.sq_moe_w4(dev(bad, "bf16"), dev(L.wr, "bf16"), 2, *L.weights(), **L.kw(), out_dtype=torch.float32)
    assert ((ids >= 0) & (ids < 8)).all()
    assert torch.isnan(y[2]).all() and torch.isnan(wts[2]).all()
    rows = [0, 1, 3, 4, 5, 6, 8]
    r_ids, r_w = P.choose(x[rows], L.wr, 2, True)
    ref, bound = L.ref(x[rows], r_ids, r_w, W_OFF)
    check(y[rows], ref, bound, "f32")


def test_padded_input_rows():
    L = Layer(7, 8, 272, 64, 32, False, "bf16")
    x = L.x(3)
    wide = torch.full((3, 320), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, 16:288] = dev(x, "bf16")
    a = sq.sq_moe_w4(wide[:, 16:288], dev(L.wr, "bf16"), 2, *L.weights(), **L.kw())
    b = sq.sq_moe_w4(dev(x, "bf16"), dev(L.wr, "bf16"), 2, *L.weights(), **L.kw())
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_one_workspace_for_many_calls_and_two_graphs():
    """Different sizes in turn, then two captured graphs that share the workspace, replayed in turn."""
    L, M = Layer(8, 8, 256, 128, 64, True, "bf16"), Layer(9, 5, 144, 80, 32, False, "f32")
    ws = sq.sq_moe_w4_workspace(64, 256, 256, 8, 8)
    runs = []
    for layer, T, k in ((L, 33, 2), (M, 1, 3), (L, 1, 1), (M, 64, 5)):
        x = layer.x(T)
        xd, wr = dev(x, layer.dt), dev(layer.wr, layer.dt)
        y = torch.empty(T, layer.D, device=DEV)

        def call(layer=layer, xd=xd, wr=wr, k=k, y=y):
            return sq.sq_moe_w4(xd, wr, k, *layer.weights(), **layer.kw(), y=y, workspace=ws)

        call()
        r_ids, r_w = P.choose(x, layer.wr, k, True)
        ref = layer.ref(x, r_ids, r_w, W_OFF)
        check(y, *ref, "f32")
        runs.append((call, y, xd, ref))
    graphs = []
    for call, y, xd, ref in runs[:2]:
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            call()
        graphs.append((g, y, ref))
    for _ in range(3):
        for g, y, ref in graphs:
            y.zero_()
            g.replay()
        torch.cuda.synchronize()
        for g, y, ref in graphs:
            check(y, *ref, "f32")


def test_two_streams_with_a_workspace_each():
    L = Layer(10, 16, 512, 256, 128, False, "bf16")
    x = [L.x(8), L.x(8)]
    xd, wr = [dev(a, "bf16") for a in x], dev(L.wr, "bf16")
    want = [sq.sq_moe_w4(a, wr, 4, *L.weights(), **L.kw())[0] for a in xd]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [sq.sq_moe_w4_workspace(8, 512, 256, 16, 4) for _ in streams]
    ys = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(30):
        for a, st, ws, y in zip(xd, streams, spaces, ys):
            sq.sq_moe_w4(a, wr, 4, *L.weights(), **L.kw(), y=y, workspace=ws, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for y, w in zip(ys, want))


def test_what_a_call_allocates_belongs_to_its_stream():
    """The current stream is busy while calls on two others make their own workspaces and choices, which are
    dropped at once: a zero-fill left to the current stream, or memory passed from one stream to the other,
    would show."""
    L = Layer(13, 16, 512, 256, 128, False, "bf16")
    xd, wr = [dev(L.x(8), "bf16") for _ in range(2)], dev(L.wr, "bf16")
    want = [sq.sq_moe_w4(a, wr, 4, *L.weights(), **L.kw()) for a in xd]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # some 50 ms
    ys = []
    for _ in range(20):
        ys.append([sq.sq_moe_w4(a, wr, 4, *L.weights(), **L.kw(), stream=st)[0] for a, st in zip(xd, streams)])
    for st in streams:
        st.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(y, w[0]) for pair in ys for y, w in zip(pair, want))
    torch.cuda._sleep(100_000_000)
    routed = sq.sq_moe_w4_routed(xd[0], want[0][1], want[0][2], *L.weights(), **L.kw(), stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(routed, want[0][0])


def test_experts_past_32_bit_offsets():
    """2.7 GB of gate and up codes; only the last experts are named."""
    E, D, F = 80, 4096, 8192
    w13 = torch.randint(0, 256, (E, 2 * F, D // 2), dtype=torch.uint8, device=DEV)
    s13 = (torch.rand(E, D // 128, 2 * F, device=DEV) * 0.002 + 0.001).to(torch.bfloat16)
    w2 = torch.randint(0, 256, (E, D, F // 2), dtype=torch.uint8, device=DEV)
    s2 = (torch.rand(E, F // 128, D, device=DEV) * 0.002 + 0.001).to(torch.bfloat16)
    rng = np.random.default_rng(11)
    x = P.bf16(rng.normal(0, 1, (2, D)).astype(np.float32))
    ids, wts = np.array([[79], [70]], np.int32), np.array([[0.5], [1.5]], np.float32)
    y = sq.sq_moe_w4_routed(dev(x, "bf16"), dev(ids), dev(wts), w13, s13, w2, s2, out_dtype=torch.float32)

    def val(w, s, K):
        return lambda e: P.values(w[e].cpu().numpy(), s[e].float().cpu().numpy(), None, K, 128)
    check(y, *P.experts(x, ids, wts, val(w13, s13, D), val(w2, s2, F), 128, 2.0 ** -16, 0.0), "f32")


def test_empty_batch_and_a_foreign_workspace():
    L = Layer(12, 4, 64, 32, 32, False, "bf16")
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device=DEV)
    y, ids, wts = sq.sq_moe_w4(x, dev(L.wr, "bf16"), 2, *L.weights(), **L.kw(), workspace=torch.zeros(256, dtype=torch.uint8, device=DEV))
    assert y.shape == (0, 64) and ids.shape == (0, 2)
    with pytest.raises(sq.SQError):
        sq.sq_moe_w4(dev(L.x(1), "bf16"), dev(L.wr, "bf16"), 2, *L.weights(), **L.kw(),
                     workspace=torch.zeros(256, dtype=torch.uint8, device=DEV))
