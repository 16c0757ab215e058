"""Arguments that the binding of the paged-cache calls refuses: a stream of another device than the tensors', and
sections that no 32-bit number holds."""
import pytest
import torch

from memory_bound_decode_qk_gb300 import edge_ops


class Elsewhere:
    """What the binding reads of a torch stream, on a device that holds none of the tensors."""
    cuda_stream = 0
    device = torch.device("cuda", 63)


def test_a_stream_of_another_device_is_refused():
    with pytest.raises(ValueError, match="cuda:63"):
        edge_ops._on(torch.device("cuda", 0), Elsewhere())


@pytest.mark.gpu
def test_calls_refuse_a_stream_of_another_device():
    i32 = dict(dtype=torch.int32, device="cuda")
    q, k = torch.zeros(2, 2, 64, device="cuda"), torch.zeros(32, 2, 64, device="cuda")
    table, lens, refs = torch.zeros(2, 4, **i32), torch.ones(2, **i32), torch.ones(4, **i32)
    one, caches = torch.zeros(1, **i32), edge_ops.PageCaches([k], 8)
    calls = [lambda s: edge_ops.paged_attention(q, k, k, table, lens, page_size=8, stream=s),
             lambda s: edge_ops.pages_copy(caches, one, one, stream=s),
             lambda s: edge_ops.pages_free(table, lens, refs, one, stream=s),
             lambda s: edge_ops.pages_fork(caches, table, lens, refs, one, one, stream=s),
             lambda s: edge_ops.pages_compact(caches, table, refs, stream=s)]
    for call in calls:
        with pytest.raises(ValueError, match="cuda:63"):
            call(Elsewhere())
    assert lens.tolist() == [1, 1] and refs.tolist() == [1] * 4


@pytest.mark.parametrize("sections", [(2 ** 32 + 8, 12, 12), (8, 12, 12 - 2 ** 32)])
def test_sections_past_32_bits_are_refused(sections):
    # as 32-bit numbers they would be 8, 12 and 12
    with pytest.raises(ValueError, match="sections"):
        edge_ops._axis_args(sections, "blocks", None, 4)
