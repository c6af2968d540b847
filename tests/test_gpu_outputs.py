"""Outputs that the cache operators allocate (needs a GPU): tensors like any of torch's, each with storage of its
own, on the stream that the call runs on."""
import numpy as np
import pytest
import torch

from cache_util import host
from paged_fp8_kv_04_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _calls(stream=None):
    mass = torch.rand(3, 2, 40, device="cuda")
    lens = torch.tensor([40, 9, 31], dtype=torch.int32, device="cuda")
    x, scores = torch.randn(3, 4, 50, device="cuda"), torch.zeros(3, 4, device="cuda")
    ends, lasts = torch.zeros(3, 4, dtype=torch.uint8, device="cuda"), torch.ones(3, 4, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    yield B.evict_select(mass, lens, budget=16, stream=stream)
    yield B.beam_select(x, scores, eos=1, finished=ends, lengths=lasts, stream=stream)
    torch.cuda.synchronize()


def test_every_output_has_storage_of_its_own():
    for outs in _calls():
        for t in outs:
            assert t.storage_offset() == 0 and t.untyped_storage().nbytes() == t.numel() * t.element_size() and t.is_contiguous()
        assert len({t.untyped_storage().data_ptr() for t in outs}) == len(outs)


def test_an_output_that_grows_leaves_the_others_as_they_are():
    for outs in _calls():
        torch.cuda.synchronize()
        before = [host(t).copy() for t in outs]
        for i, t in enumerate(outs):
            t.resize_(2 * t.numel() + 8).fill_(113)
            torch.cuda.synchronize()
            for j in range(i + 1, len(outs)):
                assert np.array_equal(host(outs[j]), before[j]), (i, j)


def test_outputs_on_a_given_stream_and_their_record():
    side = torch.cuda.Stream()
    for outs in _calls(side):
        for t in outs:
            t.record_stream(torch.cuda.current_stream())
            assert t.device == torch.device("cuda:0")
    torch.cuda.synchronize()
