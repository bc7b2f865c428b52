"""lr_fwd_diff: long rows, rows beside values that are not finite, and what the
weights' and the squares' range leave, against the fp64 definition."""
import numpy as np
import pytest
import torch

import gated_delta_rule_fwd_gb300 as lr
from oracle import attention as oa

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
BITS = {F32: 24, BF16: 8}          # half a step of the type, 2^-bits relative
NW = lr.NO_WINDOW
LR_OK = 0
EPS = 1e-6
types = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
widths = pytest.mark.parametrize("d", [32, 64, 128])


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from gated_delta_rule_fwd_gb300.build import build
    build()
    lr.device_status()
    yield torch.device("cuda:0")
    assert lr.device_status() == LR_OK


def rnd(seed, *shape, dtype=F32, std=1.0):
    g = torch.Generator("cpu").manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def np64(t):
    return t.detach().cpu().double().numpy()


def within(got, want, bound, what=""):
    got = np64(got)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} for {want[bad][0]} +- {bound[bad][0]}")


def inputs(B, H, Hk, Tq, Tk, d, dtype, seed=1):
    q, k, v = (rnd(seed + i, B, 2 * h, t, d, dtype=dtype) for i, (h, t) in enumerate(((H, Tq), (Hk, Tk), (Hk, Tk))))
    return q, k, v, 0.2 + 0.6 * torch.rand(H, generator=torch.Generator().manual_seed(seed))


@types
@widths
def test_diff_rows_of_many_tiles(dev, d, dtype):
    """Rows over up to 32 tiles, whose maxima grow along the way, so that scores, weights and
    outputs are rescaled and replaced in turn: right, and the same bits each time."""
    H, T = 2, 4096
    q, k, v, lam = inputs(1, H, 1, T, T, d, dtype, seed=301)
    k = (k.float() * torch.linspace(0.1, 3.0, T)[:, None]).to(dtype)
    ref, bound, _ = oa.diff(np64(q), np64(k), np64(v), np64(lam), NW, 0, d ** -0.5, BITS[dtype],
                            8 if dtype == BF16 else None, None, EPS)
    on = [t.to(dev) for t in (q, k, v, lam)]
    first = lr.lr_fwd_diff(*on, eps=EPS)
    within(first, ref, bound)
    for _ in range(20):
        assert torch.equal(lr.lr_fwd_diff(*on, eps=EPS), first)
