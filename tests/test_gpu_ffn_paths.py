"""GPU tests of the gated feed-forward block, the BitLinear gradients and the W8A8 product, path by
path: every kernel instance that the choices by size, alignment and type can take, values at the ends
of the range, and calls on a stream that is not the current one."""
import numpy as np
import pytest

import ffn_plain as plain
from test_gpu_ffn import _code, _f32, _layer, _np, _say, _step, _step_state, _t, dev  # noqa: F401  (dev: fixture)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------- streams
def test_buffers_of_a_given_stream_leave_queued_work_alone(dev):  # noqa: F811
    """Tensors dropped while the current stream still has work on them queued, of the sizes that calls
    on another stream then allocate: the queued work and the calls both give what they would alone."""
    torch, bl = dev
    m, k, f = 96, 512, 700
    s = _step_state(torch, bl, m, k, f, 41)
    want = [t.clone() for t in _step(torch, bl, s)]
    sizes = [4 * m * f, 4 * m * k, 4 * f * k, 4 * f * k, m * k, 4 * m, bl.bitlinear_gated_backward_workspace_size(m, k, f),
             bl.bitlinear_backward_workspace_size(m, f, k)]
    busy = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for rep in range(3):
        _say(f"dropped tensors, repetition {rep}")
        dropped = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
        out = torch.empty(4096, 4096, device="cuda")
        for _ in range(10):
            torch.mm(busy, busy, out=out)
        sums = []
        for i, t in enumerate(dropped):
            t.fill_(i + 1)
        torch.mm(busy, busy, out=out)
        for t in dropped:
            sums.append(t.to(torch.int64).sum())
        del t, dropped
        h = bl.bitlinear_gated_forward(s["x"], s["Wg"], s["ag"], s["Wu"], s["au"], s["act"], stream=side)
        dx, dwg, dwu, _, _ = bl.bitlinear_gated_backward(s["dh"], s["g"], s["u"], s["x_q"], s["beta"], s["Wg"], s["ag"],
                                                         s["Wu"], s["au"], s["act"], stream=side)
        _, dwd, _ = bl.bitlinear_backward(s["dy"], s["h_q"], s["hbeta"], s["Wd"], s["ad"], stream=side)
        torch.cuda.current_stream().wait_stream(side)
        got = [h.clone(), dx.clone(), dwg.clone(), dwu.clone(), dwd.clone()]
        # handed back to the allocator before the copies have run, and asked for again on the other stream
        del h, dx, dwg, dwu, dwd
        bl.bitlinear_gated_forward(s["x"], s["Wg"], s["ag"], s["Wu"], s["au"], s["act"], stream=side)
        torch.cuda.synchronize()
        assert [int(v) for v in sums] == [(i + 1) * n for i, n in enumerate(sizes)]
        assert all(torch.equal(a, b) for a, b in zip(got, [want[0], want[4], want[5], want[6], want[3]]))
