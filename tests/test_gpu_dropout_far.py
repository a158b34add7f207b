"""Dropout of elements past 2^34, whose block number (index / 4) needs the counter's second word."""
import numpy as np
import pytest

from oracle import experts as ox

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.slow]

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from latent_moe_layer_gb300 import experts as ex  # noqa: E402

SEED, OFFSET, FAR = 0xDEADBEEF12345678, (3 << 32) + 17, 1 << 34


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


@pytest.mark.parametrize("lead", [0, 1], ids=["pieces", "elements"])       # 16-byte pieces; rows off their boundaries
def test_mask_past_the_counter_s_first_word(lead):
    n = FAR + 1024
    if torch.cuda.mem_get_info()[0] < 2 * (n + lead) + (4 << 30):
        pytest.skip("needs 36 GB of free device memory")
    x = torch.ones(n + lead, dtype=torch.float16, device="cuda")[lead:]
    ex.dropout(x, 0.5, SEED, OFFSET, out=x)
    for lo in (0, FAR - 512, FAR, n - 512):
        i = np.arange(lo, lo + 512, dtype=np.uint64)
        assert np.array_equal(x[lo:lo + 512].double().cpu().numpy(), ox.keep_mask(i, 0.5, SEED, OFFSET) * 2.0), lo
    # a first word alone would repeat the mask of the beginning
    assert not torch.equal(x[FAR:FAR + 1024], x[:1024])
    del x
    torch.cuda.empty_cache()
