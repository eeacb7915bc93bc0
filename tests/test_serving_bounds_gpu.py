"""The serving operators (rglru_add_rmsnorm and its neighbours) at the ends of what their calls allow: counts near
2^31, probabilities far below a row's largest, waits that run out, batches that name rows twice, and the forms that
a call picks by its size.  Worlds, oracle and bars as in test_serving_gpu.py."""
import pytest
import torch

from lm_causal_depthwise_b200 import api

pytestmark = pytest.mark.gpu

dev = "cuda"
bf = torch.bfloat16


# ------------------------------------------------------------------------------------------------- add_rmsnorm
def test_add_rmsnorm_counts_rows_up_to_the_type():
    """2^31 - 1 rows: the row that a CTA would take after its last one lies past 2^31."""
    if torch.cuda.mem_get_info()[0] < 76 << 30:
        pytest.skip("needs 69 GB")
    M, N, tail = 2 ** 31 - 1, 8, 20000
    g = torch.Generator(device=dev).manual_seed(0)
    x = torch.full((M, N), 3.0, dtype=bf, device=dev)
    x[-tail:] = torch.randn((tail, N), generator=g, device=dev).to(bf)
    w = torch.arange(1, N + 1, dtype=torch.float32, device=dev) / 4
    out = torch.zeros_like(x)
    api.add_rmsnorm(x, None, w, out=out)
    last, _ = api.add_rmsnorm(x[-tail:].clone(), None, w)
    assert torch.equal(out[-tail:], last)
    row, _ = api.add_rmsnorm(x[:1].clone(), None, w)
    for i in range(0, M - tail, 1 << 27):
        part = out[i:min(i + (1 << 27), M - tail)]
        assert torch.equal(part.amin(0), row[0]) and torch.equal(part.amax(0), row[0])
