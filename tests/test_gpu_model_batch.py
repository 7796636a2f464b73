"""TrainingModel.set_batch: the batch is the model's from then on, on whichever stream."""
import pytest
import torch

from moe_routing_capacity_gb300.model import TrainingModel

from test_gpu_training_model import make_model

pytestmark = pytest.mark.gpu

I32 = torch.int32


def batch(m, ids):
    cu = torch.tensor([0, 100, 250], device="cuda", dtype=I32)
    pos = torch.cat([torch.arange(100), torch.arange(156)]).to("cuda", I32)
    return ids.clone(), cu, pos


def test_the_callers_tensors_may_take_the_next_batch():
    """ids and positions overwritten between set_batch and the step: lookup, angles and the
    table's gradient are those of the batch that was set."""
    m, ids, entries, teacher, weight = make_model()
    want = {n: t.clone() for n, t in m.step(entries, teacher, weight).items()}
    loss = m.loss.clone()
    mine, cu, pos = batch(m, ids)
    m.set_batch(mine, cu, pos)
    mine.copy_((mine + 5) % m.vocab)
    pos.zero_()
    got = m.step(entries, teacher, weight)
    assert torch.equal(m.loss, loss)
    for n in want:
        assert torch.equal(got[n], want[n]), n


def test_a_batch_of_other_shapes_or_types_is_refused():
    m, ids, *_ = make_model()
    mine, cu, pos = batch(m, ids)
    for bad in (pos[:1], pos[None]):
        with pytest.raises(ValueError, match="pos"):
            m.set_batch(mine, cu, bad)
    with pytest.raises(TypeError, match="pos"):
        m.set_batch(mine, cu, pos.long())
    with pytest.raises(ValueError, match="ids"):
        m.set_batch(mine[:5], cu, pos)
    m.set_batch(mine, cu, None)                     # positions 0, 1, ...
    assert all(b.pos is None for b in m.blocks)


def test_the_first_batch_on_another_stream_than_the_models():
    """The model is made on a stream that is still busy, its first batch set and run on
    another: what making it queued (a plan of no words, a cleared status) comes first."""
    m, ids, entries, teacher, weight = make_model()
    want = {n: t.clone() for n, t in m.step(entries, teacher, weight).items()}
    mine, cu, pos = batch(m, ids)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(100_000_000)                  # some 50 ms
    late = TrainingModel(m.blocks, m.w, embed_scale=m.embed_scale)
    late.set_batch(mine, cu, pos, stream=side)
    for _ in range(2):
        got = late.step(entries, teacher, weight, stream=side)
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(got[n], want[n]), n
        assert int(late.status) == 0
