"""The norm gradient over many steps: its CTAs stay and take rows in turn, with
a ring of two or four stages of copies ahead, pointers that advance over rows
and heads, and sums of the parameters' gradients carried along.  Row counts here
make every CTA go round its ring more than once and leave the last step part
empty; head counts do not divide a step, so the heads wrap at another place
each time."""
import re

import pytest
import torch

import audio_video_flow_gb300 as h3
from test_gpu_train_ops import DTYPES, KINDS, norm_rows, ok, run_norm

pytestmark = pytest.mark.gpu

STAGES = 4   # of the longer ring

# rows, heads, width: per-head rows of 4 to 32 threads in one and two chunks,
# then whole-CTA rows of one, three and four chunks per thread
SHAPES = [(31000, 7, 8), (17000, 7, 64), (9000, 7, 128), (7150, 7, 129), (10001, 3, 300), (5003, 3, 500), (1501, 5, 520),
          (1303, 7, 1030), (4703, 1, 2688), (881, 7, 2300), (3209, 1, 5376), (1607, 1, 8190)]


def steps_of_last_call():
    info = h3.h3_last_kernel_info()
    units, per_step, ctas = (int(re.search(k + r"=(\d+)", info).group(1)) for k in (" rows", "rows/step", "ctas"))
    return units, per_step * ctas


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("rows, heads, width", SHAPES)
def test_many_steps(kind, dtype, rows, heads, width):
    run_norm(kind, dtype, rows, heads, width)
    units, step = steps_of_last_call()
    assert units == rows * heads
    # more steps than stages, the last one not whole
    assert units > (STAGES + 1) * step and units % step, (units, step)
    assert heads == 1 or step % heads, (step, heads)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("rows, heads, width", [(9000, 7, 128), (5003, 3, 500), (1501, 5, 520), (4703, 1, 2688), (1607, 1, 8190)])
def test_many_steps_in_place_and_in_short_calls(kind, dtype, rows, heads, width):
    """dx over dy or over x while later rows are being copied in, and the rows
    a few at a time, each CTA one step: the same bits.  Without the parameters'
    gradients too."""
    tdtype, code, _ = DTYPES[dtype]
    cfg = h3.make_norm_config(KINDS[kind], width, code, code)
    x, dy = (norm_rows(rows, heads, width, tdtype, s) for s in (1, 2))
    gain = torch.rand(width, generator=torch.Generator().manual_seed(3)).to(tdtype).cuda()
    rs, hs = x.stride(0), x.stride(1)
    ws = torch.empty(h3.h3_norm_backward_workspace_bytes(cfg, rows, heads), dtype=torch.uint8, device="cuda")

    def run(n, x, dy, dx, params=True):
        dg, db = (torch.empty(width, device="cuda") for _ in range(2)) if params else (None, None)
        h3.h3_norm_backward(cfg, n, heads, x, rs, hs, gain, dy, rs, hs, dx, rs, hs, dg, db, ws if params else None)
        return dg, db

    dx = torch.empty_like(x)
    dg, db = run(rows, x, dy, dx)
    _, step = steps_of_last_call()
    over_dy, over_x, alone, parts = dy.clone(), x.clone(), torch.empty_like(x), torch.empty_like(x)
    dg1, db1 = run(rows, x, over_dy, over_dy)
    dg2, db2 = run(rows, over_x, dy, over_x)
    run(rows, x, dy, alone, params=False)
    few = step // heads
    for r in range(0, rows, few):
        run(min(few, rows - r), x[r:], dy[r:], parts[r:], params=False)
    ok()
    for other in (over_dy, over_x, alone, parts):
        assert torch.equal(other[..., :width], dx[..., :width])
    assert torch.equal(dg1, dg) and torch.equal(db1, db) and torch.equal(dg2, dg) and torch.equal(db2, db)
