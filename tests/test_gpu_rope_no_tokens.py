"""The weights' gradients of a rotation's backward without tokens: sums of nothing, as an empty microbatch leaves them."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [8, 64, 80, 128])
@pytest.mark.parametrize("rot", [0, 8])
def test_weights_gradients_without_tokens(d, rot):
    import bit_nf4_quantised_amd as nf4
    q, k = (torch.empty(0, h, d, dtype=torch.bfloat16, device="cuda:0") for h in (4, 2))
    w, pos, rope = torch.ones(d, dtype=torch.bfloat16, device="cuda:0"), torch.empty(0, dtype=torch.int64, device="cuda:0"), nf4.Rope(rot)
    for both in (True, False):
        for accumulate in (False, True):
            dw = torch.full((3, 128), float("nan"), device="cuda:0")
            nf4.qlora_rope_bwd(rope, pos, q, k, q, k, q=q, k=k, q_weight=w, k_weight=w, dq_weight=dw[0, :d] if both else None,
                               dk_weight=dw[1, :d], accumulate=accumulate)
            torch.cuda.synchronize()
            assert torch.all(dw[1, :d].isnan() if accumulate else dw[1, :d] == 0)
            assert torch.all(dw[0, :d].isnan() if accumulate or not both else dw[0, :d] == 0)
            assert torch.all(dw[:2, d:].isnan()) and torch.all(dw[2].isnan())      # nothing else


def test_without_tokens_from_a_graph():
    import bit_nf4_quantised_amd as nf4
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda:0")
    w, dw, rope = torch.ones(64, dtype=torch.bfloat16, device="cuda:0"), torch.full((64,), 2.0, device="cuda:0"), nf4.Rope(0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nf4.qlora_rope_bwd(rope, None, q, None, q, None, q=q, q_weight=w, dq_weight=dw)
    for _ in range(3):
        dw.fill_(2.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.all(dw == 0)
