"""The norm's variants that depend on the number of rows and on wide rows, with
the bounds of tests/test_gpu_rmsnorm.py: more rows than the grid holds at once, the
most elements per thread, rings of one and two CTAs per SM that go round."""
import pytest
import torch

import gated_delta_rule_37_gb300 as gdr
from tests.test_gpu_rmsnorm import BF, E4, F, check_fwd, make, run_fwd
from tests.test_gpu_rmsnorm import test_bwd as backward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdr.load()


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,D", [(80000, 128), (40000, 136), (2600, 4096), (1300, 8192), (700, 16384), (3000, 1001),
                                 (400, 8199), (160, 20001)])
def test_fwd(M, D, dtype):
    c = make(M + D, M, D, dtype)
    check_fwd(c, *run_fwd(c, residual=True, y_dtype=dtype), residual=True)
    for group in (0, 32, 128):
        check_fwd(c, *run_fwd(c, residual=group != 0, y_dtype=E4, group=group), residual=group != 0, group=group)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,D", [(1300, 4104), (1300, 5120), (1000, 7168), (1300, 8192), (700, 8200), (700, 16384),
                                 (700, 16392), (3000, 136), (2500, 504), (30000, 40), (700, 8199)])
def test_bwd(M, D, dtype):
    backward(M, D, dtype)
