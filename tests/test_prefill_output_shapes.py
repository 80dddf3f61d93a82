"""prefill_chunk and prefill_expanded write [N, H, dim] and [N, H]: outputs of as
many values in another order are refused, not filled in that order."""
import pytest
import torch

import mla_paged_decode_gb300 as mla
from chunk_cases import SCALE, ints

N, H = 6, 4


def wrong(device):
    """(out, lse) for a dim, one of them laid out otherwise."""
    def pairs(dim):
        out, lse = torch.zeros(N, H, dim, dtype=torch.bfloat16, device=device), torch.zeros(N, H, device=device)
        for shape in ((H, N, dim), (N, H * dim), (N * H, dim), (1, N, H, dim), (N, dim, H), (N + 1, H, dim), (N, H, dim // 2)):
            yield torch.zeros(shape, dtype=torch.bfloat16, device=device), lse
        for shape in ((H, N), (N * H,), (N, H, 1), (1, N, H), (N, H + 1)):
            yield out, torch.zeros(shape, device=device)
    return pairs


@pytest.mark.parametrize("dim", [512, 128])
def test_the_check(dim):
    q = torch.zeros(N, H, 576, dtype=torch.bfloat16)
    ws = torch.zeros(256, dtype=torch.uint8)
    good = torch.zeros(N, H, dim, dtype=torch.bfloat16), torch.zeros(N, H)
    assert mla._prefill_outputs(*good, q.device, N, H, dim, ws, None, q) is ws
    for out, lse in wrong("cpu")(dim):
        with pytest.raises(ValueError, match="must be \\[N, H"):
            mla._prefill_outputs(out, lse, q.device, N, H, dim, ws, None, q)


@pytest.mark.gpu
def test_the_calls():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_paged_decode_gb300 import build
    build.build()
    bf16 = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    kv, table, lens, starts = bf16(2, 64, 576), ints([[1, 0]]), ints([70]), ints([0, N])
    for out, lse in wrong("cuda")(512):
        with pytest.raises(ValueError):
            mla.prefill_chunk(bf16(N, H, 576), kv, table, lens, starts, SCALE, 0, out, lse)
    for out, lse in wrong("cuda")(128):
        with pytest.raises(ValueError):
            mla.prefill_expanded(bf16(N, H, 192), bf16(9, H, 128), bf16(9, 64), bf16(9, H, 128), starts, ints([0, 9]), True,
                                 SCALE, 0, out, lse)
