"""The router and its gradient against the 64-bit definition."""

import numpy as np
import pytest
import torch

import dispatch_grouped_gemm_amd as moe
import ops_ref as ref
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def shape_of(T, E, K):
    return moe.MoeShape(T=T, H=128, I=128, K=K, E_total=E, E_local=min(E, 512))


def run(logits, K, renorm):
    T, E = logits.shape
    s = shape_of(T, E, K)
    ids = torch.full((T, K), 77, dtype=torch.int32, device=DEV)
    w = torch.full((T, K), 77.0, device=DEV)
    moe.moe_route(s, logits, ids, w, renormalize=renorm)
    return s, ids, w


def check_forward(logits, K, renorm, ids, w):
    """ids equal; weights within the float32 error of exp (1 ulp, and the rounding of
    l - m, which moves exp by |l - m| 2^-24), of a sum of at most 16 + 6 additions per
    lane, and of one division."""
    rid, rw, p, reach = ref.route(logits, K, renorm)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    off = rw * (ref.U32 * (2 * reach + 40))[:, None] + 2.0 ** -149
    ref.assert_close(w, rw, off, "weights")
    return p, reach


def draw(T, E, dt, seed, pads=True):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(T, E, generator=g) * 2
    if pads and T > 3:
        l[1] = float("-inf")                      # a row with nothing to choose
        l[2, 1:] = float("-inf")                  # one expert left
        l[3] = torch.finfo(dt).min                # a mask of the type's lowest value
    return l.to(dt).to(DEV)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dt", [BF, HF, F32])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (5, 8, 8), (7, 6, 8), (33, 63, 2), (16, 64, 1),
                                   (16, 65, 3), (9, 129, 6), (130, 384, 6), (17, 513, 4),
                                   (11, 1024, 8)])
def test_route(T, E, K, dt, renorm):
    say("route", T, E, K, dt, renorm)
    logits = draw(T, E, dt, seed=T * 1000 + E)
    s, ids, w = run(logits, K, renorm)
    p, reach = check_forward(logits, K, renorm, ids, w)
    g = torch.randn(T, K, generator=torch.Generator().manual_seed(5)).to(DEV)
    # slots of -1 carry weights and gradients that must not count
    g = torch.where(ids < 0, float("nan"), g)
    w2 = torch.where(ids < 0, float("nan"), w)
    dl = torch.full((T, E), 77.0, dtype=dt, device=DEV)
    moe.moe_route_backward(s, logits, ids, w2, g, dl, renormalize=renorm)
    d, mag = ref.route_backward(ids, w, p, g, E, renorm)
    # the products and the sum of K terms, and p's own error where it is recomputed
    ref.assert_close(dl, d, mag * (ref.U32 * (2 * reach + 60))[:, None] + 2.0 ** -149, "dlogits")
    if renorm:
        dl2 = torch.full_like(dl, 77.0)
        moe.moe_route_backward(s, None, ids, w2, g, dl2, renormalize=True)
        assert torch.equal(dl2, dl)


@pytest.mark.parametrize("dt", [BF, HF, F32])
def test_ties_take_the_lower_expert(dt):
    l = torch.zeros(6, 384)
    l[1] = torch.arange(384) % 7
    l[2, ::2] = -0.0                              # equal to +0
    l[3, 200:] = 1.0
    l[4] = -torch.arange(384) // 100
    l[5, 383] = l[5, 0] = l[5, 64] = 3.0
    logits = l.to(dt).to(DEV)
    for renorm in (True, False):
        _, ids, w = run(logits, 8, renorm)
        check_forward(logits, 8, renorm, ids, w)
    assert ids[0].tolist() == list(range(8)) and ids[2].tolist() == list(range(8))


@pytest.mark.parametrize("renorm", [True, False])
def test_infinities_and_nan(renorm):
    inf, nan = float("inf"), float("nan")
    l = torch.randn(6, 40, generator=torch.Generator().manual_seed(1))
    l[0, 5] = inf
    l[1, [3, 30]] = inf                           # share the weight
    l[2, ::2] = nan
    l[3] = nan
    l[4, 1:] = -inf
    l[5, 7] = 3e38
    l[5, 8] = -3e38
    logits = l.to(DEV)
    _, ids, w = run(logits, 4, renorm)
    clean = torch.where(torch.isnan(logits), -inf, logits)
    check_forward(clean, 4, renorm, ids, w)
    assert ids[3].tolist() == [-1] * 4 and w[3].tolist() == [0.0] * 4
    assert w[1, :2].tolist() == [0.5, 0.5] and w[0].tolist() == [1.0, 0.0, 0.0, 0.0]


def test_gradient_against_differences():
    """The gradient in float64 differences of the 64-bit weights: a step of 1e-6 leaves
    about 1e-6 of curvature and 1e-10 of rounding; the kernel's float32 adds 1e-6."""
    T, E, K = 4, 12, 3
    l = torch.randn(T, E, dtype=torch.float64, generator=torch.Generator().manual_seed(2))
    l = l.float().double()
    g = torch.randn(T, K, generator=torch.Generator().manual_seed(3))
    for renorm in (True, False):
        s, ids, w = run(l.float().to(DEV), K, renorm)
        dl = torch.empty(T, E, device=DEV)
        moe.moe_route_backward(s, l.float().to(DEV), ids, w, g.to(DEV), dl, renormalize=renorm)
        h = 1e-6
        for e in range(E):
            up, dn = l.clone(), l.clone()
            up[:, e] += h
            dn[:, e] -= h
            fu, fd = ((ref.route(v, K, renorm)[1] * g.double()).sum(1) for v in (up, dn))
            assert torch.allclose(dl[:, e].cpu().double(), (fu - fd) / (2 * h), rtol=0, atol=1e-5)


def test_many_tokens_and_a_captured_graph():
    T, E, K = 20011, 384, 6
    s = shape_of(T, E, K)
    logits = torch.empty(T, E, dtype=BF, device=DEV)
    ids = torch.empty(T, K, dtype=torch.int32, device=DEV)
    w = torch.empty(T, K, device=DEV)
    g = torch.randn(T, K, device=DEV)
    dl = torch.empty_like(logits)
    logits.normal_()

    def step():
        moe.moe_route(s, logits, ids, w, renormalize=False)
        moe.moe_route_backward(s, logits, ids, w, g, dl, renormalize=False)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        logits.normal_()
        ids.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        got = [ids.clone(), w.clone(), dl.clone()]
        step()
        for u, v in zip(got, (ids, w, dl)):
            assert torch.equal(u, v)
    pick = torch.arange(0, T, 1777)
    check_forward(logits[pick.to(DEV)], K, False, ids[pick.to(DEV)], w[pick.to(DEV)])


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dt", [BF, HF, F32])
def test_logits_off_16_byte_borders(dt, renorm):
    """Logits and gradients that start one element into a buffer, and what lies around."""
    T, E, K = 50, 384, 6
    say("route off borders", dt, renorm)
    logits = torch.empty(T * E + 1, dtype=dt, device=DEV)[1:].view(T, E)
    logits.copy_(draw(T, E, dt, seed=3))
    assert logits.data_ptr() % 16 and logits.is_contiguous()
    s, ids, w = run(logits, K, renorm)
    p, reach = check_forward(logits, K, renorm, ids, w)
    g = torch.randn(T, K, generator=torch.Generator().manual_seed(6)).to(DEV)
    g = torch.where(ids < 0, float("nan"), g)
    room = torch.full((T * E + 2,), 7.0, dtype=dt, device=DEV)
    dl = room[1:-1].view(T, E)
    moe.moe_route_backward(s, logits, ids, w, g, dl, renormalize=renorm)
    d, mag = ref.route_backward(ids, w, p, g, E, renorm)
    ref.assert_close(dl, d, mag * (ref.U32 * (2 * reach + 60))[:, None] + 2.0 ** -149, "dlogits")
    assert float(room[0]) == 7.0 and float(room[-1]) == 7.0


@pytest.mark.parametrize("dt", [BF, HF])
def test_every_16_bit_pattern(dt):
    """Every value of the type, both zeros and every NaN, in shuffled rows."""
    say("route patterns", dt)
    bits = np.random.default_rng(11).permutation(1 << 16).astype(np.uint16).view(np.int16)
    logits = torch.from_numpy(bits).view(dt).view(2048, 32).to(DEV)
    logits[0] = float("nan")
    logits[1] = -float("nan")
    logits[2, ::2], logits[2, 1::2] = 0.0, -0.0
    for renorm in (True, False):
        s, ids, w = run(logits, 8, renorm)
        rid = ref.route(logits, 8, renorm)[0]
        np.testing.assert_array_equal(ids.cpu().numpy(), rid)


@pytest.mark.parametrize("dt", [BF, HF, F32])
@pytest.mark.parametrize("E", [128, 384, 1024])
def test_the_largest_side_by_side(E, dt):
    """All the chosen in neighbouring experts or 16 apart, falling, rising and equal."""
    say("route side by side", E, dt)
    T, K = 48, 8
    l = torch.randn(T, E, generator=torch.Generator().manual_seed(E)) * 0.25
    for t in range(T):
        step = (1, 16, 8 * 16)[t % 3]
        at = [(t + step * i) % E for i in range(10)]
        l[t, at] = torch.tensor([[4.0 - 0.25 * i for i in range(10)],
                                 [4.0 + 0.25 * i for i in range(10)],
                                 [4.0] * 10][t // 3 % 3])
    logits = l.to(dt).to(DEV)
    for renorm in (True, False):
        s, ids, w = run(logits, K, renorm)
        check_forward(logits, K, renorm, ids, w)
