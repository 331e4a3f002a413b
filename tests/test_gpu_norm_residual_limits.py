"""The norms at the widths where their kernels change: the widest rows that one CTA, two and four of a cluster take, and
the next ones, in each type and direction (the checks are those of test_gpu_norm_residual)."""
import pytest
import test_gpu_norm_residual as N
import torch

pytestmark = pytest.mark.gpu
B16, H16, F = torch.bfloat16, torch.float16, torch.float32

# s, b, h, tp, dtype, post, pre, gate, scale, checkpoint
FORWARD = [
    (5, 1, 16384, 1, H16, True, True, "column", 0.5, False),
    (3, 1, 16392, 1, B16, True, True, "none", 0.5, True),
    (3, 1, 32776, 1, H16, True, True, "column", 0.5, True),
    (2, 1, 65536, 1, B16, True, True, "none", 0.5, True),
    (2, 1, 65544, 1, B16, True, True, "none", 0.5, True),
    (4, 1, 8200, 1, F, True, True, "column", 0.5, True),
    (3, 1, 16392, 1, F, True, True, "column", 0.5, False),
    (3, 1, 32768, 1, F, True, True, "none", 0.5, True),
    (2, 1, 32776, 1, F, True, True, "none", 0.5, True),
]
BACKWARD = [
    (6, 1, 8192, 1, B16, True, True, "column", 0.5, True),
    (6, 1, 8200, 1, H16, True, True, "column", 0.5, True),
    (5, 1, 16384, 1, B16, True, True, "column", 0.5, False),
    (5, 1, 16392, 1, H16, True, True, "none", 0.5, True),
    (4, 1, 32768, 1, B16, True, True, "column", 0.5, True),
    (4, 1, 32776, 1, B16, True, True, "column", 0.5, True),
    (6, 1, 4104, 1, F, True, True, "column", 0.5, True),
    (6, 1, 6144, 1, F, True, True, "column", 0.5, False),
    (6, 1, 6152, 1, F, True, True, "none", 0.5, True),
    (5, 1, 8200, 1, F, True, True, "column", 0.5, True),
    (4, 1, 16384, 1, F, True, True, "column", 0.5, True),
    (4, 1, 16392, 1, F, True, True, "column", 0.5, True),  # four CTAs would need more than 512 threads each
    (4, 1, 16392, 1, F, True, True, "none", 0.5, False),
]


def _id(c):
    return f"{c[2]}-{str(c[4])[6:]}{'-c8' if c[9] else ''}"


@pytest.mark.parametrize("case", FORWARD, ids=_id)
def test_forward_at_the_limits(cuda_lib, case):
    N.test_forward(cuda_lib, case, False)


@pytest.mark.parametrize("case", BACKWARD, ids=_id)
def test_backward_at_the_limits(cuda_lib, case):
    N.test_backward(cuda_lib, case, False)
