"""The grouped bf16 products on every tile (train_shapes.py), against whole numbers bit for bit."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

from test_train_gpu import check_matmul, gen  # noqa: E402
from train_shapes import CASES  # noqa: E402


@pytest.mark.parametrize("way,M,N,K,G", [(w,) + c for w in CASES for c in CASES[w]])
def test_matmul_of_every_tile(way, M, N, K, G):
    """Groups of any length, some empty, rows in front of the first and behind the last."""
    ends = None
    if G > 1:
        ends = [1] + torch.randint(1, M - 7, (G - 1,), generator=gen(M + G)).sort().values.tolist() + [M - 7]
    check_matmul(way, M, N, K, ends, out="bf16", add=G % 2 == 0)
    check_matmul(way, M, N, K, ends, out="f32", add=G % 2 == 1)
