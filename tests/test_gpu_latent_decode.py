"""The example that runs the operators with the swap-in path, as a user would."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.mark.parametrize("e4m3", [True, False])
def test_latent_decode_example(e4m3):
    from hierarchical_kv_cache_hs_gb300.examples import latent_decode as ex
    got = ex.run(e4m3=e4m3)
    assert got["errors"] == 0
    # every step: 64 recent tokens (resident once appended, prompt rows before), the rest random
    assert got["misses"] > 0 and got["hits"] > 0
    # bf16 results of bf16 queries: two roundings (weights, output) for the decode, four (keys,
    # values, weights, output) for the prompt, each at most half a step of 2^-8, in the 2-norm
    assert got["decode"] <= 1.5 * 2 ** -8
    assert got["prompt"] <= 2.5 * 2 ** -8
