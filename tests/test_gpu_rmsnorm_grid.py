"""The norm and its backward pass with a small grid, at widths whose rows take a whole
workgroup of eight waves: a workgroup then goes from one group of rows to the next, and
results are the same bits as with a workgroup to each."""
import pytest
import torch

import zero_sharded_optimizer_zr_amd as zr
from gpu_util import device, say
from test_gpu_rmsnorm import backward, check_backward, check_forward, data, forward, rstd_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,cols", [(90, 4097), (90, 5000), (600, 5000), (90, 8192), (40, 8193), (40, 11008), (530, 11008),
                                       (40, 16384)])
def test_rows_of_a_whole_workgroup(monkeypatch, rows, cols, dtype):
    """One round to a group of rows (an odd number: the next group begins at once) and, past
    512 rows, two in some groups and one in the others."""
    device()
    x, res, w, dy, dh = data(rows, cols, dtype, cols + rows)
    rstd = rstd_of(x)

    def run():
        out = forward(x, w, res)
        check_forward(out, x, w, res)
        grads = backward(dy, x, w, rstd, dh)
        check_backward(grads, dy, x, w, rstd, dh)
        return [out[k].contiguous().view(torch.uint8).clone() for k in ("h", "y", "q", "s")] + \
               [out["rstd"].clone()] + [t.clone() for t in grads]

    say(rows, cols, dtype)
    full = run()
    for cap in ("8", "9", "24"):
        monkeypatch.setenv("ZR_MAX_GRID", cap)
        assert all(torch.equal(a, b) for a, b in zip(run(), full)), cap
