"""A completion that the int8 GEMM signals in both CTAs of a pair must be one
that the second CTA waits for before it leaves: an arrival on its way to the
shared memory of a CTA that has exited is undefined.  Read from the source; the
second CTA's copying warp waits for `empty`, its epilogue for `accfull`, and the
last completion (`drain`) is for the issuing CTA alone."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_only_quantized_rtn_b200", "csrc")


def test_the_second_cta_waits_for_what_is_signalled_to_it():
    src = open(os.path.join(CSRC, "int8_gemm.cuh")).read()
    both = set(re.findall(r"mma_commit_pair_both_on\(on, &?(\w+)", src))
    assert both == {"empty", "accfull"}
    assert re.findall(r"mma_commit_pair_on\(on, &?(\w+)", src) == ["drain"]


@pytest.mark.gpu
def test_pairs_back_to_back():
    """Many pair launches one behind the other, their CTAs leaving while the next ones start; exact sums each time."""
    import torch
    import weight_only_quantized_rtn_b200 as m

    g = torch.Generator().manual_seed(2)
    M, N, K = 520, 4096, 384
    xq, wq = (torch.randint(-127, 128, (n, K), generator=g, dtype=torch.int8).cuda() for n in (M, N))
    one = torch.ones(N, device="cuda")
    want = (xq.double() @ wq.double().t()).float()  # below 2^24: exact in fp32
    ys = [torch.full((M, N), float("nan"), device="cuda") for _ in range(40)]
    for y in ys:
        m.int8_linear_into(y, xq, one[:M], wq, one)
    m.check_status()
    assert all(torch.equal(y, want) for y in ys)
