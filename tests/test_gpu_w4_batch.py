"""The batch kernel of the 4-bit product where its buffers go round: many tiles to a cluster, every cluster size, sums
that are exact, so that every bit must agree with the integers'."""
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


@pytest.mark.parametrize("M,K,dt", [(20, 1024, "bf16"), (32, 4096, "bf16"), (32, 8208, "bf16"), (64, 1040, "bf16"),
                                    (64, 2048, "bf16"), (64, 4096, "bf16"), (12, 2064, "f32"), (32, 2048, "f32"),
                                    (130, 4096, "bf16")])
def test_every_tile_of_a_cluster_is_exact(M, K, dt):
    """Codes, zero points, x and scales are small integers: the sums stay below 2^24, whatever their order.  Neighbouring
    tiles differ, so a sum that came into a buffer before it was read, or was read before it came, shows."""
    rng = np.random.default_rng(M + K)
    N = 24840
    codes = rng.integers(0, 16, (N, K)).astype(np.uint8)
    sg = (2.0 ** rng.integers(0, 3, (-(-K // 128), N))).astype(np.float32)
    zp = rng.integers(0, 16, sg.shape).astype(np.uint8)
    wq = P.pack(codes)
    x = rng.integers(-3, 4, (M, K)).astype(np.float32)
    w = P.values(wq, sg, zp, K, 128)
    assert 15 * 4 * 3 * K < 2 ** 24
    ref = torch.from_numpy(x).to(DEV).double() @ dev(w).T
    xd, wqd, sgd, zpd = dev(x, dt), dev(wq), dev(sg, "bf16"), dev(zp)
    y = [torch.empty(M, N, device=DEV) for _ in range(4)]
    for _ in range(5):
        for t in y:
            sq.sq_w4_gemm(xd, wqd, sgd, zpd, y=t)
    assert all(torch.equal(t.double(), ref) for t in y)
    assert sq.sq_device_error() == 0
