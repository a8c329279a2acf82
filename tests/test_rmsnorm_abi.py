"""Host-side checks of pqg_rmsnorm_quant (CPU only: nothing is launched)."""
import pytest

from precision_activation_quantization_b200 import pqg
from test_abi import FAKE, host_only

INV, UNS, ALN = pqg.PQG_ERR_INVALID_ARG, pqg.PQG_ERR_UNSUPPORTED, pqg.PQG_ERR_ALIGNMENT


def at(i):
    return FAKE + (i << 32)


def call(**kw):
    a = dict(in_ptr=at(0), residual_ptr=at(1), weight_ptr=at(2), residual_out_ptr=at(3),
             out_ptr=at(4), scales_ptr=at(5), global_scale_ptr=None, M=4, K=256, group=128,
             eps=1e-6, in_dtype=pqg.PQG_BF16, out_dtype=pqg.PQG_E4M3,
             scale_fmt=pqg.PQG_SCALE_FP32, scale_layout=pqg.PQG_ROW_MAJOR, stream=None)
    a.update(kw)
    return pqg.pqg_rmsnorm_quant(**a)


@host_only
@pytest.mark.parametrize("kw,status", [
    (dict(in_dtype=2), INV), (dict(out_dtype=0), INV), (dict(scale_fmt=3), INV),
    (dict(scale_layout=4), INV), (dict(group=0), INV), (dict(M=-1), INV), (dict(K=200), INV),
    (dict(eps=-1e-6), INV), (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV),
    (dict(in_ptr=0), INV), (dict(weight_ptr=0), INV), (dict(out_ptr=0), INV),
    (dict(scales_ptr=0), INV), (dict(global_scale_ptr=at(6)), INV),
    (dict(scale_fmt=pqg.PQG_SCALE_E4M3, out_dtype=pqg.PQG_E2M1, group=16), INV),   # no g
    (dict(scale_fmt=pqg.PQG_SCALE_E4M3, group=16, global_scale_ptr=at(6)), UNS),   # e4m3 codes
    (dict(group=256, K=512), UNS), (dict(K=16512), UNS), (dict(K=16400, group=16400), UNS),
    (dict(out_dtype=pqg.PQG_INT8, scale_fmt=pqg.PQG_SCALE_UE8M0), UNS),
    (dict(out_dtype=pqg.PQG_E2M1), UNS), (dict(scale_layout=pqg.PQG_UE8M0_PACKED), UNS),
    (dict(in_ptr=at(0) + 16), ALN), (dict(residual_ptr=at(1) + 8), ALN),
    (dict(weight_ptr=at(2) + 16), ALN), (dict(residual_out_ptr=at(3) + 2), ALN),
    (dict(out_ptr=at(4) + 8), ALN), (dict(scales_ptr=at(5) + 2), ALN),
    (dict(scale_fmt=pqg.PQG_SCALE_E4M3, out_dtype=pqg.PQG_E2M1, group=16,
          global_scale_ptr=at(6) + 1), ALN),
    (dict(residual_out_ptr=at(1) + 512), INV),          # overlaps the residual in part
    (dict(residual_out_ptr=at(2)), INV),                # the weight
    (dict(out_ptr=at(0)), INV), (dict(out_ptr=at(3)), INV), (dict(scales_ptr=at(2)), INV),
    (dict(scales_ptr=at(4) + 16), INV),
])
def test_rejects_before_launch(kw, status):
    before = pqg.pqg_launch_count()
    assert call(**kw) == status
    assert pqg.pqg_launch_count() == before


@host_only
def test_zero_rows_is_ok_and_launches_nothing():
    before = pqg.pqg_launch_count()
    assert call(M=0, in_ptr=0, out_ptr=0, scales_ptr=0) == pqg.PQG_OK
    assert pqg.pqg_launch_count() == before
