"""sf_sync_status: what it reports, and what it costs (GPU)."""

import statistics
import time

import pytest
import torch

from layer_optimizer_gb300 import native

pytestmark = pytest.mark.gpu


def _median(f, n=300):
    times = []
    for _ in range(n):
        t = time.perf_counter()
        f()
        times.append(time.perf_counter() - t)
    return statistics.median(times)


def test_an_error_is_reported_once_and_again_when_it_happens_again():
    side = torch.cuda.Stream()
    for stream in (None, side):
        native.sf_test_device_wait_runs_out(100_000, stream=stream)
        with pytest.raises(native.SfError, match="ran out"):
            native.sf_sync_status(stream)
        native.sf_sync_status(stream)
        native.sf_sync_status()


def test_it_costs_a_few_copies_whatever_the_library_has():
    # all its error words wait together: a copy of each (nine now) would be nine of these, or 84 us where one call takes 21
    x = torch.zeros(1, device="cuda")
    native.sf_sync_status()
    assert _median(native.sf_sync_status) < 5 * _median(lambda: x.cpu())
