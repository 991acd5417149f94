"""Products of 8-bit integers in large tiles, of every height and number of row blocks, against the
definition in 64 bits (tolerances as in test_gpu_int8)."""
import pytest

import int8_cases as cases
import test_gpu_int8 as int8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,K,N", [c[:3] for c in cases.LINEAR])
@pytest.mark.parametrize("name", ["none", "swiglu"])
def test_linear_in_large_tiles(T, K, N, name):
    int8.test_linear(T, K, N // 2 if name == "swiglu" else N, name)


@pytest.mark.parametrize("T,k,E,cap,K,N", [c[:6] for c in cases.EXPERTS])
@pytest.mark.parametrize("name", ["gelu", "swiglu"])
def test_experts_in_large_tiles(T, k, E, cap, K, N, name):
    int8.test_experts(T, k, E, cap, 0.0, K, N // 2 if name == "swiglu" else N, name)
