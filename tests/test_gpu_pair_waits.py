"""The bounded waits of the kernels that run on pairs of CTAs (vsf_ns_gemm, the
experts' products): a pipeline that stands still ends with an error word, its copies
landed and its tensor memory free, and the calls behind it are right."""
import time

import pytest
import torch

pytestmark = pytest.mark.gpu

MS = 1_000_000
# Tiles that the leading and the other CTA of a pair load (-1: all): the other one up
# to a ring of stages ahead, the leading one, neither, from the first tile on and later.
STALLS = [(0, -1), (1, -1), (2, -1), (1, 1), (-1, 0), (2, 1)]


@pytest.fixture
def limits():
    from fsdp_buffer_layout_gb300 import vsf as V
    try:
        yield V.vsf_selftest_pair_waits
    finally:
        torch.cuda.synchronize()
        V.vsf_selftest_pair_waits()


def stalled(limits, lead, other, call):
    """Runs call() on a pipeline that stands still; how long it took."""
    torch.cuda.synchronize()
    limits(20 * MS, lead, other)
    t0 = time.perf_counter()
    call()
    torch.cuda.synchronize()
    seconds = time.perf_counter() - t0
    limits()
    # a few limits and sleeps; and 2 s, where the leading CTA has loaded more
    ahead = 0 <= other and (lead < 0 or other < lead)
    assert (0.018 if not ahead else 1.9) <= seconds < (1.0 if not ahead else 4.0), seconds


@pytest.mark.parametrize("kind", ["forward", "backward_input", "backward_weight"])
@pytest.mark.parametrize("lead,other", STALLS)
def test_products_that_stand_still(limits, kind, lead, other):
    from fsdp_buffer_layout_gb300.experts import ExpertLinear
    g = torch.Generator(device="cuda").manual_seed(3)
    # 22 tiles of lanes, an expert's rows in two tiles of three stages, or in five
    # stages of which the last one is mended
    counts, n, k = [300, 310, 0, 290, 300, 7, 300, 311, 300], 5600, 192
    if kind == "backward_input":
        n, k = k, n
    starts = torch.tensor([sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int32, device="cuda")
    x, d_y = (torch.randn(sum(counts), w, device="cuda", generator=g).bfloat16() for w in (k, n))
    w = torch.randn(len(counts), n, k, device="cuda", generator=g).bfloat16()
    args = {"forward": (x, w, starts), "backward_input": (d_y, w, starts), "backward_weight": (d_y, x, starts)}[kind]
    op, still = (ExpertLinear(sum(counts), len(counts), n, k) for _ in range(2))
    want = getattr(op, kind)(*args).clone()
    assert op.device_error() == 0
    stalled(limits, lead, other, lambda: getattr(still, kind)(*args))
    assert still.device_error() == 2
    for _ in range(3):
        assert torch.equal(getattr(op, kind)(*args), want)
    assert op.device_error() == 0


@pytest.mark.parametrize("lead,other", STALLS)
def test_newton_schulz_products_that_stand_still(limits, lead, other):
    from fsdp_buffer_layout_gb300 import vsf as V
    g = torch.Generator(device="cuda").manual_seed(4)
    m, n, k = 4096, 3840, 320
    a, b = (torch.randn(rows, k, device="cuda", generator=g).bfloat16() for rows in (m, n))
    err = torch.zeros(2, dtype=torch.int32, device="cuda")

    def product(at):
        d = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
        V.vsf_ns_gemm(a_mn=False, b_mn=False, sym=False, M=m, N=n, K=k, batch=1, A=a.data_ptr(), lda=k,
                      sa=m * k, B=b.data_ptr(), ldb=k, sb=n * k, alpha=1.0, beta=0.0, C=None, ldc=n, sc=m * n,
                      D=d.data_ptr(), ldd=n, sd=m * n, d_err=err[at:].data_ptr(),
                      stream=torch.cuda.current_stream().cuda_stream)
        return d

    want = product(0)
    stalled(limits, lead, other, lambda: product(1))
    assert torch.equal(product(0), want) and err.tolist() == [0, 2]


def signs(rows, width, seed):
    """-1, 0 and 1: their products' sums are exact in fp32 up to 2^24 of them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-1, 2, (rows, width), device="cuda", generator=g).bfloat16()


@pytest.mark.parametrize("counts,n,k,limit", [
    ([(1 << 21) + 5], 64, 64, 2 * MS),               # a tile of 32769 stages, the last one mended
    ([1 << 18, 37, 0, 21], 2048, 2048, MS // 2),     # long tiles in front of the mended ones
    ([(1 << 20) + 16], 130, 70, MS)])
def test_long_tiles_are_not_given_up(limits, counts, n, k, limit):
    """A wait for a whole tile, or for the next mended stage, is longer than the limit
    while stages go by: the limit counts from the last of them."""
    from fsdp_buffer_layout_gb300.experts import ExpertLinear
    rows, experts = sum(counts), len(counts)
    starts = torch.tensor([sum(counts[:i]) for i in range(experts + 1)], dtype=torch.int32, device="cuda")
    # rows start on 16-byte boundaries
    x, d_y = (signs(rows, -(-w // 8) * 8, w + i)[:, :w] for i, w in enumerate((k, n)))
    op = ExpertLinear(rows, experts, n, k)
    op.backward_weight(d_y, x, starts)
    limits(limit)
    d_w = op.backward_weight(d_y, x, starts)
    assert op.device_error() == 0
    cuts = starts.tolist()
    for e, (a, b) in enumerate(zip(cuts, cuts[1:])):
        want = d_y[a:b].float().t() @ x[a:b].float()
        assert torch.equal(d_w[e], want.bfloat16()), e


def test_a_long_depth_is_not_given_up(limits):
    """The same for the other products: 2^15 stages a tile."""
    from fsdp_buffer_layout_gb300.experts import ExpertLinear
    rows, depth = 40, 1 << 21
    starts = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    x, w = signs(rows, depth, 1), signs(64, depth, 2)[None]
    op = ExpertLinear(rows, 1, 64, depth, with_grad=False)
    limits(2 * MS)
    y = op.forward(x, w, starts)
    assert op.device_error() == 0
    assert torch.equal(y, (x.float() @ w[0].float().t()).bfloat16())
    flip = ExpertLinear(rows, 1, depth, 64, with_grad=False)
    out = torch.empty(rows, 64, dtype=torch.bfloat16, device="cuda")
    d_x = flip.backward_input(x, w[0].t().contiguous()[None], starts, out=out)
    assert flip.device_error() == 0 and torch.equal(d_x, y)
