"""The experts' layer on a part of the SMs leaves the others alone."""
import pytest
import torch

import combine_ep_get_02_gb300 as ep
from test_gpu_layer import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("calls", [1, 2])
def test_the_other_sms_stay_free(calls):
    """A long call on half of the SMs, whose CTAs leave no shared memory of an SM to others, and beside it, on another stream,
    a short one on the other half: it ends while the long one's first kernel, two thirds of its work, still runs."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    long = Case(ep, 64, 64, 8, 4096, 2048, num_sms=sms // 2)
    short = Case(ep, 16, 4, 2, 512, 256, num_sms=sms // 2)
    want = long.run(), short.run()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    start, long_end, short_end = (torch.cuda.Event(enable_timing=True) for _ in range(3))
    outs = [torch.empty_like(w) for w in want]
    for _ in range(3):
        torch.cuda.synchronize()
        with torch.cuda.stream(streams[0]):
            start.record()
            for _ in range(calls):
                long.run(out=outs[0])
            long_end.record()
        with torch.cuda.stream(streams[1]):
            streams[1].wait_event(start)
            for _ in range(calls):
                short.run(out=outs[1])
            short_end.record()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
        assert start.elapsed_time(short_end) < start.elapsed_time(long_end) / 2
