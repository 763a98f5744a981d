"""The embedding gradient at every length of its chunks of sorted positions (8,
16, 32 and 64, by the work there is), around whole chunks and with runs of one id
from none to all of them.  Gradients are small integers, whose sums are exact in
fp32; bf16 results are those rounded once."""
import pytest
import torch

from nonlinear_rnn_solve_pararnn_amd import api
from tests.gpu_helpers import DEV, say
from tests.test_gpu_embedding import ids_of

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
KINDS = ["uniform", "frequent", "same", "two"]


def check(N, V, D, kind, dtype, shift=0):
    gen = torch.Generator().manual_seed(N + D)
    T = TYPES[dtype]
    room = torch.zeros(N * D + shift, dtype=T, device=DEV)
    values = torch.randint(-8, 9, (N, D), generator=gen, dtype=torch.int8)
    grad = room[shift:].view(N, D).copy_(values)
    ids = ids_of(N, V, kind, N + 1)
    # exact in fp32: sums of N integers of at most 8
    want = 2.0 * torch.zeros(V, D).index_add_(0, ids.cpu(), values.float())
    out = torch.full((V * D + shift,), float("nan"), dtype=T, device=DEV)[shift:].view(V, D)
    say("embedding gradient", N, V, D, kind, dtype, shift)
    got = api.embedding_backward(ids, grad, V, scale=2.0, out=out)
    assert torch.equal(got.cpu(), want.to(T))
    for _ in range(2):
        assert torch.equal(api.embedding_backward(ids, grad, V, scale=2.0), got)


# chunks of 8: whole ones, one more, one less; then of 16, 32 and 64 (with 256 CUs)
EIGHT = [7, 8, 9, 15, 16, 17, 64, 65, 512, 513, 2047, 4096, 4097, 8191]
LONGER = [16384, 16385, 16399, 131072, 131073, 131103, 262144, 262145, 262207]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("N", EIGHT)
def test_short_chunks(N, kind):
    check(N, 37, 40, kind, "f32")
    check(N, 37, 31, kind, "bf16", shift=1)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("N", LONGER)
def test_longer_chunks(N, kind, dtype):
    check(N, 300, 8, kind, dtype)
    check(N, 70000, 11, kind, dtype, shift=3)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["frequent", "two"])
@pytest.mark.parametrize("N,D", [(17024, 4100), (33025, 4104), (33023, 4099)])
def test_longer_chunks_of_wide_rows(N, D, kind, dtype):
    """Several column blocks: 32 positions a chunk at 17024 x 4100, 64 at 33000 x 4100."""
    check(N, 200, D, kind, dtype, shift=D % 2)
