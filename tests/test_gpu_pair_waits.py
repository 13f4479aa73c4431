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
