"""Products of 65 to 256 tokens, two to four groups of 64, at the columns' lengths from which each
form is taken; bit for bit against the definition."""
import pytest
import torch

from serving_ref import DTYPES, IDS
from test_gpu_wcols import inputs, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("K", [2560, 2561, 3200, 3201, 5000])
@pytest.mark.parametrize("M", [65, 128, 129, 191, 193, 256])
def test_groups_of_tokens(M, K, dtype):
    """A few columns' tiles, so that runs of the list end inside them and groups have runs of their own."""
    same(*inputs(M, K, 300 + M, dtype, M + K), relu=bool(M % 2))


@pytest.mark.parametrize("M", [129, 192, 256])
def test_one_tile_of_columns(M):
    """Fewer blocks than runs."""
    for K, N in ((4000, 1), (4000, 100), (3300, 129)):
        same(*inputs(M, K, N, torch.float16, N))
