"""Rotary positions far out against angles in 60 decimal digits that know nothing of the table of steps."""
import math
from decimal import Decimal

import pytest
import torch

dlo = pytest.importorskip("layerwise_weight_offload_slot_gb300")

from test_gpu_packed import U, float32_by_default, stream, within  # noqa: E402,F401
from test_packed_rope_table import FACTOR, FAST, LENGTH, SLOW, TWO_PI, frequencies  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda"
ENDS = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 12345, -2 ** 31 + 999, 1 << 30, -(1 << 29) + 7, 123456789, -98765432, 1 << 24, 65535, -1, 0, 1]


@pytest.mark.parametrize("back", [False, True], ids=["forward", "backward"])
@pytest.mark.parametrize("layout", [dlo.ROPE_INTERLEAVED, dlo.ROPE_HALF], ids=["interleaved", "half"])
@pytest.mark.parametrize("scaling", range(5))
@pytest.mark.parametrize("dim,theta", [(128, 10000.0), (44, 500000.0)])
def test_angles_at_the_ends_of_int32(dim, theta, scaling, layout, back):
    """The result's rounding, U, sine, cosine and products, 2^-20 of (|u| + |v|), and the angle's error: 2^-26 of a turn and
    2^-52 (blended: 2^-51) |position|, times 2 pi (|u| + |v|)."""
    r = dlo.make_rope(heads=1, head_dim=128, ldx=128, ldy=128, layout=layout,
                      axes=[dict(dim=dim, theta=theta, scaling=scaling, factor=FACTOR, length=LENGTH, fast=FAST, slow=SLOW)])
    steps = torch.from_numpy(dlo.dlo_rope_steps(r)).to(DEV)
    rows, n = len(ENDS), dim // 2
    x = torch.randn((rows, 128), generator=torch.Generator(device=DEV).manual_seed(dim), device=DEV).to(torch.bfloat16)
    y = torch.empty_like(x)
    positions = torch.tensor(ENDS, dtype=torch.int32, device=DEV)
    call = dlo.dlo_op_rope_bwd if back else dlo.dlo_op_rope_fwd
    call(r, x.data_ptr(), positions.data_ptr(), steps.data_ptr(), rows, y.data_ptr(), stream())
    f = [v / TWO_PI for v in frequencies(dim, theta, scaling)]
    turns = [[float((Decimal(at) * v) % 1) for v in f] for at in ENDS]
    angle = torch.tensor(turns, dtype=torch.float64, device=DEV) * (-2 * math.pi if back else 2 * math.pi)
    i = torch.arange(n, device=DEV)
    u, v = (2 * i, 2 * i + 1) if layout == dlo.ROPE_INTERLEAVED else (i, i + n)
    a, b = x.double()[:, u], x.double()[:, v]
    want, bound = x.double().clone(), torch.full((rows, 128), 1e-30, dtype=torch.float64, device=DEV)
    want[:, u], want[:, v] = a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()
    table = 2.0 ** (-52 if scaling < dlo.ROPE_BY_TURNS else -51)
    turn = 2.0 ** -26 + table * positions.double().abs()[:, None]
    size = (a.abs() + b.abs()) * (2.0 ** -20 + 2 * math.pi * turn)
    bound[:, u] += size
    bound[:, v] += size
    within(y, want, bound + U * want.abs(), "y")
