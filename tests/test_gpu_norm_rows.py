"""Norms of many rows, the kernels in which a block takes several or shares its SM, against 64 bits."""

import pytest

import memory_bound_gemv_gb300 as mbg

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from test_gpu_decode import BF16, F16, F32, check_norm, no_device_error, normal  # noqa: E402,F401

# rows and widths on both sides of the rules: several rows per block, staged operands, two blocks per SM, odd widths
SHAPES = [(2000, 4096), (5000, 1024), (3000, 2048), (700, 8192), (160, 9216), (400, 14336), (1300, 14336), (200, 16000),
          (1400, 333), (4000, 777), (1400, 4001), (700, 8191), (400, 9001), (153, 10241), (400, 11908), (608, 12001),
          (1400, 11908), (400, 15001), (320, 20000)]


@pytest.mark.parametrize("rows,width", SHAPES)
@pytest.mark.parametrize("yt,xt,ht", [(BF16, BF16, BF16), (F32, F32, F16), (F32, F16, F32)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_many_rows(rows, width, yt, xt, ht, kind):
    y, x = normal(111, (rows, width), yt, 1.7), normal(112, (rows, width), xt, 3.0)
    one = lambda i, t=xt: 1 + normal(i, (width,), F32, 0.2).to(t)  # noqa: E731
    check_norm(y, x, ht, kind=kind, post=True, post_weight=one(1), gate=normal(2, (width,), xt, 0.5), alpha=0.7,
               pre_weight=one(3), pre_bias=normal(4, (width,), F32, 0.3), eps=1e-5)  # shared operands
    if rows * width <= 10 ** 7:
        row = lambda i, t=xt: normal(i, (rows, width), t, 0.3)  # noqa: E731
        check_norm(y, x, ht, kind=kind, gate=row(5), pre_weight=row(6), pre_bias=row(7, F16), unit_offset=True)
        check_norm(y, x, ht, kind=kind, post=True, post_weight=one(1, F32), gate=row(5), pre_weight=one(3))
