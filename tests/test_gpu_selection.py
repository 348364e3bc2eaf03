"""The alternatives' selection under load, again and again: ids are whole numbers, so they are equal or wrong."""
import pytest
import torch

from speculative_decoding_verify_decode_gb300 import native

from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()


# Pieces of no more segments (of 512 logits) than alternatives are asked for, whose list of segments is not cut: of a row over
# many CTAs, of rows in one piece each with four of them on an SM, of a last piece that ends inside a segment.
@pytest.mark.parametrize("rows,vocab,top", [(1, 151936, 32), (5, 32000, 32), (608, 4096, 8), (1216, 4096, 32), (700, 16384, 32), (640, 5001, 20),
                                            (900, 500, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_alternatives_of_few_segments_every_time(dtype, rows, vocab, top):
    gen = torch.Generator(device="cuda").manual_seed(rows + vocab)
    x = (torch.randn(rows, vocab, generator=gen, device="cuda") * 4).to(dtype)
    want = torch.sort(x.float(), dim=1, descending=True, stable=True)[1][:, :top].int()
    ws = torch.empty(max(16, native.sd_logprobs_workspace_size(rows, vocab, top)), dtype=torch.uint8, device="cuda")
    ids = torch.empty(100, rows, top, dtype=torch.int32, device="cuda")
    best, status = torch.empty(rows, top, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    for i in range(len(ids)):
        native.sd_logprobs(x, top_ids=ids[i], top_logprobs=best, workspace=ws, dev_status=status)
    assert int(status) == 0 and torch.isfinite(best).all()
    wrong = (ids != want).any(-1).nonzero()
    assert len(wrong) == 0, wrong[:5].tolist()
