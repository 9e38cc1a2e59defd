"""The scored route plan around the sizes where its kernels change: k from the
candidates' range to the search over all keys, and batches of fewer and of more
chunks of 32 tokens than the GPU has SMs. Reference and tolerances are
test_gpu_route_scored's."""
import pytest

from test_gpu_route_scored import _compare, _normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,k", [(896, 17), (896, 20), (1000, 24), (300, 24), (300, 25), (256, 24), (33, 24)])
@pytest.mark.parametrize("T", [5, 130])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_k_around_the_candidates_limit(E, k, T, sigmoid):
    bias = 0.05 * _normal(1, E, 11)[0] * (1.0 if sigmoid else 0.02)
    _compare(_normal(T, E, E + T), k, bias, sigmoid=sigmoid, scale=2.5)


@pytest.mark.parametrize("T", [4863, 4865, 5001])
@pytest.mark.parametrize("E,k", [(48, 6), (290, 8)])
def test_chunks_around_the_number_of_sms(T, E, k):
    _compare(_normal(T, E, T), k, 0.05 * _normal(1, E, 12)[0], sigmoid=True, scale=1.0)
