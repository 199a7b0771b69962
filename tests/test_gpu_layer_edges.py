"""Norm gradients on the GPU at the borders of how their rows are dealt to
workgroups and teams of waves, against the plain reference in float64 within
test_gpu_layer.py's bounds."""
import pytest

from group_wise_affine_quantize_amd import _binding as B
from test_gpu_layer import check_norm_grad, gpu, norm_inputs, normal, strided  # noqa: F401  (gpu: the fixture)

pytestmark = pytest.mark.gpu


# one to eight teams; a workgroup per gate, several, a part of one; few rows under one
# gate, whose teams take them by turns
@pytest.mark.parametrize("rows,gates", [(1, "channel"), (3, "channel"), (8, "channel"), (15, "channel"), (15, 0), (15, 3), (16, 2),
                                        (35, 5), (63, 21), (510, 170), (600, 60), (1400, 200), (1200, 40)])
@pytest.mark.parametrize("dim,dt,pdt", [(96, "bf16", "f32"), (512, "f32", "bf16"), (777, "bf16", "bf16"), (1600, "f32", "f32"),
                                        (2504, "bf16", "f32"), (8200, "bf16", "bf16")])
def test_norm_gradient_however_rows_are_dealt(rows, gates, dim, dt, pdt):
    if rows * dim > 2_000_000:
        rows, gates = 210, 70       # as many rows of a wide matrix as the reference takes quickly
    t = norm_inputs(200, rows, dim, dt, pdt, True, gates, True)
    o = {"scale": 0.7, "offset": 1.0, "eps": 1e-6}
    dh_out, dz = normal(210, (rows, dim), dt), strided(normal(211, (rows, dim), dt))
    h_out, _ = B.nq_block_norm(**t, **o)
    check_norm_grad(t, h_out, dh_out, dz, B.nq_block_norm_grad(h_out, t["y"], dh_out, dz, t["post"], t["gate"], t["pre"], **o), o)
