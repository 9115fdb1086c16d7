"""The adapters' term where 16 bits of x A^T do not do, and where values are not finite."""

import pytest
import torch

import dispatch_grouped_gemm_amd as moe
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16

# rows, N and H for each way through the projection on 256 CUs: 16, 32, 64 and 128 rows
# at most; tiles in parts of H, one deep workgroup a CU, two, the largest tiles
SIZES = [(1, 72, 512), (16, 136, 512), (40, 64, 512), (64, 1000, 512), (100, 264, 512),
         (300, 520, 512), (200, 11000, 2176), (1300, 4096, 512), (4111, 4104, 512)]


def project(x, w, base, ids, a, b, scale=None):
    (T, H), (L, N, r) = x.shape, b.shape
    s = moe.AdapterShape(T=T, H=H, N=N, L=L, rank=r)
    ws = moe.alloc_adapter_workspace(s, DEV)
    ws.fill_(255)
    out = torch.full((T, N), 7.0, dtype=x.dtype, device=DEV)
    moe.moe_adapter_project(s, x, w, ids, a, b, scale, out, ws, base=base)
    return out


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("T,N,H", SIZES)
def test_all_24_bits_of_v(T, N, H, dt):
    """v0 = n, a whole number of 24 bits, and v1 = -n without its last 8: their sum, n mod 256,
    is left of them only if both products are exact.  Every sum is one of whole numbers
    below 2^24 (times a power of two that fits the type), so it is exact in float32."""
    say("24 bits", T, N, dt)
    L, r = 3, 16
    unit = 1.0 if dt is BF else 2.0 ** -12
    g = torch.Generator().manual_seed(T)
    n = torch.randint(1 << 23, 1 << 24, (T,), generator=g)
    n[0] = (1 << 24) - 1
    bit = torch.arange(24)
    x = torch.zeros(T, H)
    x[:, :24] = (n[:, None] >> bit & 1) * 2.0 ** bit * unit
    a, b = torch.zeros(L, r, H), torch.zeros(L, N, r)
    for l in range(L):
        a[l, 3 + l, :24], a[l, 11 - l, 8:24] = 1.0, -1.0
        b[l, :, 3 + l] = b[l, :, 11 - l] = 2.0 ** l
    ids = torch.randint(-1, L, (T,), generator=g)
    ids[0] = L - 1
    want = torch.where(ids >= 0, (n % 256) * 2.0 ** ids * unit, 0.0)[:, None].expand(T, N)
    x, a, b = (t.to(dt).to(DEV) for t in (x, a, b))
    zero = torch.zeros(N, H, dtype=dt, device=DEV), torch.zeros(T, N, dtype=dt, device=DEV)
    for w, base in ((zero[0], None), (None, zero[1])):
        out = project(x, w, base, ids.to(torch.int32).to(DEV), a, b)
        assert torch.equal(out.cpu(), want.to(dt)), w is not None


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("T,N,H", SIZES)
def test_small_values_beside_large_ones(T, N, H, dt):
    """A row of v holds 2^25, which B does not use, and k 2^-20, which it multiplies by 2^12:
    k 2^-8 (k of 8 bits) is exact in both types."""
    say("small beside large", T, N, dt)
    L, r = 2, 24
    g = torch.Generator().manual_seed(T)
    k = torch.randint(0, 256, (T,), generator=g)
    x = torch.zeros(T, H)
    x[:, 5], x[:, 77] = 2.0 ** 10, k * 2.0 ** -10
    a, b = torch.zeros(L, r, H), torch.zeros(L, N, r)
    a[:, 2, 5], a[:, 17, 77], b[:, :, 17] = 2.0 ** 15, 2.0 ** -10, 2.0 ** 12
    ids = torch.randint(0, L, (T,), generator=g).to(torch.int32).to(DEV)
    want = (k * 2.0 ** -8)[:, None].expand(T, N).to(dt)
    x, a, b = (t.to(dt).to(DEV) for t in (x, a, b))
    zero = torch.zeros(N, H, dtype=dt, device=DEV), torch.zeros(T, N, dtype=dt, device=DEV)
    for w, base in ((zero[0], None), (None, zero[1])):
        out = project(x, w, base, ids, a, b)
        assert torch.equal(out.cpu(), want), w is not None


def same(got, want):
    """Equal, infinities by sign and NaN as NaN."""
    got, want = got.cpu().double(), want.double()
    return bool(((got == want) | (got.isnan() & want.isnan())).all())


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("r", [16, 72])
@pytest.mark.parametrize("T,N,H", SIZES)
def test_infinities_and_nan_as_the_definition_has_them(T, N, H, r, dt):
    """Whole numbers (every finite sum is exact, and below 2^8, so the outputs are too) with
    infinities and NaN in B, in A and in x: finite times infinite, infinite times
    infinite and 0 times infinite come out as in the definition, row by row."""
    say("infinities", T, N, r, dt)
    L = 5
    inf, nan = float("inf"), float("nan")
    g = torch.Generator().manual_seed(T + r)
    whole = lambda *shape: torch.randint(-1, 2, shape, generator=g).float()
    x, w, a = torch.zeros(T, H), torch.zeros(N, H), whole(L, r, H)
    b, base = whole(L, N, r), whole(T, N)
    x[:, :8], w[:, 1:5] = whole(T, 8), whole(N, 4)
    b[:, :, 8:] *= (torch.rand(L, N, r - 8, generator=g) < 0.1)
    # adapter 0 finite; 1: one infinity in every third column; 2: two, of either sign; 3:
    # an infinite row of A, times all of B; 4: all of B infinite, and a NaN
    b[1, ::3, 5], b[2, ::2, r - 1], b[2, ::3, 3] = inf, -inf, inf
    a[3, 2, 6], b[4] = inf, inf * b[4].sign().where(b[4] != 0, torch.ones(()))
    b[4, 1, 0] = nan
    ids = torch.randint(-1, L, (T,), generator=g)
    ids[0] = 2
    if T > 8:
        x[5, 7], x[6, 6], x[7, 7] = inf, -inf, nan      # (columns that w does not use)
        ids[5:8] = torch.tensor([0, 1, 0])
    d = torch.zeros(T, N, dtype=torch.float64)
    for l in range(L):
        at = ids == l
        v = x[at].double() @ a[l].double().t()
        d[at] = v @ b[l].double().t()
    x, w, a, b, base = (t.to(dt).to(DEV) for t in (x, w, a, b, base))
    xw = x.cpu().double()
    xw[:, 5:] = 0                                       # 0 times what x holds there
    idd = ids.to(torch.int32).to(DEV)
    # x W^T has 0 times infinity in rows 5 to 7, so they are compared with a given base
    plain = torch.ones(T, dtype=torch.bool)
    plain[5:8] = False
    out = project(x, w, None, idd, a, b)
    assert same(out[plain.to(DEV)], (xw @ w.cpu().double().t() + d)[plain])
    assert same(project(x, None, base, idd, a, b), base.cpu().double() + d)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("T", [2, 40, 100, 300])
def test_rows_without_an_adapter_are_the_base_to_the_bit(T, dt):
    """-0 and subnormals among them, whatever the adapters of their neighbours."""
    say("base bits", T, dt)
    H, N, L, r = 256, 136, 3, 16
    g = torch.Generator().manual_seed(T)
    rn = lambda *shape: torch.randn(*shape, generator=g).to(dt).to(DEV)
    base = rn(T, N)
    base[:, ::3], base[:, 1::7] = -0.0, torch.finfo(dt).smallest_normal / 4
    ids = torch.randint(-1, L, (T,), generator=g).to(torch.int32)
    ids[0], ids[1] = -1, 0
    ids = ids.to(DEV)
    out = project(rn(T, H), None, base, ids, rn(L, r, H), rn(L, N, r))
    bits = lambda t: t[ids < 0].view(torch.int16)
    assert torch.equal(bits(out), bits(base))


@pytest.mark.parametrize("T,N", [(5, 72), (48, 1000), (300, 520), (1025, 264)])
def test_base_in_place(T, N):
    """out over base: a wavefront reads its next columns of base before it writes."""
    say("base in place", T, N)
    H, L, r = 512, 4, 40
    g = torch.Generator().manual_seed(T)
    rn = lambda *shape: torch.randn(*shape, generator=g).to(BF).to(DEV)
    x, a, b, base = rn(T, H), rn(L, r, H), rn(L, N, r), rn(T, N)
    ids = torch.randint(-1, L, (T,), generator=g).to(torch.int32).to(DEV)
    want = project(x, None, base, ids, a, b)
    s = moe.AdapterShape(T=T, H=H, N=N, L=L, rank=r)
    moe.moe_adapter_project(s, x, None, ids, a, b, None, base, moe.alloc_adapter_workspace(s, DEV),
                            base=base)
    assert torch.equal(base, want)


@pytest.mark.parametrize("weight", [True, False])
@pytest.mark.parametrize("T,H,N", [(262000, 8192, 8),         # x ends just below 2^32 bytes
                                   (20000, 128, 120000)])    # out and base past them
def test_offsets_past_32_bits(T, H, N, weight):
    """Whole numbers, so that every sum is exact; rows all over x and out."""
    say("offsets", T, H, N, weight)
    L, r = 3, 8
    g = torch.Generator(device=DEV).manual_seed(T)
    small = lambda *shape: torch.randint(-1, 2, shape, generator=g, device=DEV).to(BF)
    x = torch.zeros(T, H, dtype=BF, device=DEV)
    x[:, :32], x[:, -32:] = small(T, 32), small(T, 32)
    w, base, a, b = small(N, H), None, small(L, r, H), small(L, N, r)
    if not weight:
        w, base = None, torch.empty(T, N, dtype=BF, device=DEV).random_(0, 9, generator=g)
    ids = torch.randint(-1, L, (T,), generator=g, device=DEV).to(torch.int32)
    out = project(x, w, base, ids, a, b)
    at = torch.cat([torch.arange(0, T, T // 97), torch.tensor([T - 1])]).to(DEV)
    xs, got = x[at].cpu().double(), out[at].cpu().double()
    want = base[at].cpu().double() if w is None else xs @ w.cpu().double().t()
    of = ids[at].cpu()
    for l in range(L):
        want[of == l] += (xs[of == l] @ a[l].cpu().double().t()) @ b[l].cpu().double().t()
    assert torch.equal(got, want.to(BF).double())


@pytest.mark.parametrize("T,H,N", [(1, 2048, 1024), (100, 1024, 2048), (600, 1024, 1024)])
def test_two_calls_at_once(T, H, N):
    """Two streams, a workspace each, shared weights: the bits of one call after the other."""
    say("two at once", T, H, N)
    L, r = 6, 32
    g = torch.Generator().manual_seed(T)
    rn = lambda *shape: torch.randn(*shape, generator=g).to(BF).to(DEV)
    w, a, b = rn(N, H), rn(L, r, H), rn(L, N, r)
    s = moe.AdapterShape(T=T, H=H, N=N, L=L, rank=r)
    calls = []
    for _ in range(2):
        ids = torch.randint(-1, L, (T,), generator=g).to(torch.int32).to(DEV)
        calls.append((rn(T, H), ids, torch.empty(T, N, dtype=BF, device=DEV),
                      moe.alloc_adapter_workspace(s, DEV), torch.cuda.Stream()))
    want = [project(x, w, None, ids, a, b) for x, ids, _, _, _ in calls]
    torch.cuda.synchronize()
    for _ in range(10):
        for x, ids, out, ws, st in calls:
            moe.moe_adapter_project(s, x, w, ids, a, b, None, out, ws, stream=st)
    torch.cuda.synchronize()
    for (_, _, out, _, _), v in zip(calls, want):
        assert torch.equal(out, v)
