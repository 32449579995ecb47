"""The differential anchor at lengths that leave the lanes of a warp different work: rows behind the
last query or key in each quarter of the last tile, in whole units, split ones and cut streams."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from tests.test_gpu_diff_anchor import compare, dev, make  # noqa: E402


@pytest.mark.parametrize("dtype, d", [("bf16", 128), ("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("keys", [90, 2049])
@pytest.mark.parametrize("N", [5, 31, 33, 63, 97, 129, 143, 175, 200, 255])
def test_rows_of_the_last_tile(dtype, d, N, keys):
    x = make(1, N, keys, 1, d, dtype, 1000 + N + keys)
    compare(x, dev(x, dtype), 1, dtype, lens=[keys - 1])


@pytest.mark.parametrize("dtype, d", [("bf16", 128), ("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("keys", [5, 31, 33, 97, 143, 175])
def test_rows_of_the_last_key_tile(dtype, d, keys):
    x = make(2, 1200, keys, 1, d, dtype, 2000 + keys)
    compare(x, dev(x, dtype), 1, dtype, lens=[keys, keys // 2])
