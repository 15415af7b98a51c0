"""GPU tests of the budgeted special stream and of the 8-bit cache where the calls meet unusual
state: reported timeouts, infinite keys, long records, evictions of many streams."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import oracle  # noqa: E402
import workloads as wl  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


def work(**kw):
    base = dict(name="edges", num_blocks=1, num_streams=1, num_heads=2, head_dim=64, page_size=256,
                patches_per_frame=200, specials_per_frame=6, scale_frames=1, sliding_window=2,
                frames=6, dtype="bf16", value_scale=1.0)
    base.update(kw)
    return wl.Workload(**base)


def harness(w, kind, **kw):
    from budget_harness import Stream
    return Stream(w, kind, **kw)


# ---------------------------------------------------------------- accumulated weights

@pytest.mark.parametrize("kind", ["e4m3", "bf16", "f32"])
def test_a_reported_timeout_adds_nothing(kind):
    """The status word as a wait that gave up leaves it (set from the host): the running totals stay
    as they are until the report has been read."""
    from budget_harness import to_device
    import streaming_paged_kv_two_gb300 as spk
    w = work(frames=8)
    h = harness(w, kind)
    h.track()
    for f in range(w.frames):
        h.append(f)
    n = w.frames * w.specials_per_frame
    q = h.queries(6, 1)
    h.cache.plan_rows(6, h.ws, h.st)
    lse = torch.from_numpy(h.oracle(0, q, 6)[1].astype(np.float32)).cuda()
    qd = to_device(q, h.w.dtype)
    h.weights[:, :n] = 0.5
    h.ws.view(torch.int32)[0] = 1
    h.cache.accumulate_weights(0, qd, lse, h.ws, h.st)
    torch.cuda.synchronize()
    assert torch.equal(h.weights[:, :n], torch.full_like(h.weights[:, :n], 0.5))
    with pytest.raises(spk.SpkError) as e:
        h.status()
    assert e.value.code == spk.SPK_ERR_DEVICE_TIMEOUT
    h.cache.accumulate_weights(0, qd, lse, h.ws, h.st)
    torch.cuda.synchronize()
    assert float(h.weights[:, :n].min()) > 0.5
    assert h.status() == 0
    h.close()
