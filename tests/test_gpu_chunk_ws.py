"""What the chunk attention's workspace held before a call does not matter, whatever it is."""
import pytest
import torch

from test_gpu_chunk import Case, status
from test_gpu_paged import BF16, E8M0, S128

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def fill(ws, what):
    if what == "zeros":
        ws.zero_()
    elif what == "ones":
        ws.fill_(0xFF)
    else:  # 64-bit words that rise: behind each array of first rows lie smaller ones than behind that of last rows
        n = ws.numel() // 8
        ws[:8 * n].view(torch.int64).copy_(torch.arange(n, device="cuda") * (1 if what == "rising" else -1))


@pytest.mark.parametrize("what", ["rising", "falling", "zeros", "ones"])
@pytest.mark.parametrize("dtype,page,B", [(S128, 64, 3), (E8M0, 16, 5), (BF16, 8, 2), (E8M0, 64, 32), (S128, 64, 64)])
def test_copied_rows_end_with_zeros_of_no_sequence(what, dtype, page, B):
    """The rows of zeros behind the last sequence's are found without a look at any sequence's place."""
    new, hist = [11] * B if B > 8 else [60 + i for i in range(B)], [17 * i for i in range(B)]
    new[-1], hist[-1] = new[-1] + 1, hist[-1] + 130
    c = Case(B, dtype, 64, page, new, hist)
    fill(c.ws, what)
    torch.cuda.synchronize()
    c.call()
    assert status() == 0
    c.check(only=range(0, 62, 7))
