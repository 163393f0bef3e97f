"""The forward's loop over rows: more rows than the groups of warps of a launch, at each length class
(1, 2, 4 and 8 warps a row, each number of groups a lane) and for each source (bf16, fp32, a
checkpoint), so that every group refills its slot; and each class' lengths with few rows. Against
the oracle, within the tolerances of test_gpu_norm."""
import pytest

import test_gpu_norm

pytestmark = pytest.mark.gpu

# 148 SMs by 24 groups of one warp, 12 or 8 of two, 6 or 4 of four, 3 or 2 of eight: two or three rounds
MANY = [(9700, 264), (9700, 512), (9700, 1000), (5000, 1032), (3700, 2048), (3000, 2056), (2500, 4096),
        (1300, 4104), (1300, 6152), (1300, 8192), (700, 8200), (700, 12296), (500, 16384)]


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("rows,d", MANY)
def test_forward_many_rows(rows, d, dtype, wdtype, kind):
    test_gpu_norm.test_forward(rows, d, dtype, wdtype, kind)


@pytest.mark.parametrize("rows,d,dtype", [(9700, 264, "f32"), (9700, 264, "bf16"), (3700, 2048, "bf16"),
                                          (2500, 4096, "f32"), (700, 8200, "bf16")])
def test_forward_saves_and_reads_a_checkpoint_many_rows(rows, d, dtype):
    test_gpu_norm.test_norm_saves_and_reads_a_checkpoint(rows, d, dtype, "layer")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d", [(7, 2056), (148, 520), (7, 4096), (149, 4096), (7, 6152), (3, 12296)])
def test_forward_few_rows(rows, d, dtype):
    test_gpu_norm.test_forward(rows, d, dtype, dtype, "layer")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d", [(3, 72), (2000, 72), (2000, 104), (5000, 128), (40, 136)])
def test_backward_short_lane_classes(rows, d, dtype):
    test_gpu_norm.test_backward(rows, d, dtype, "f32", "layer")
