"""A Routing given to gemm_route_scored has all five tensors, or the call is refused before anything runs."""
import pytest

torch = pytest.importorskip("torch")

from dense_fp16_gemm_03_gb300 import build as pkg_build  # noqa: E402
from dense_fp16_gemm_03_gb300 import ragged as R  # noqa: E402


def routing(rows, experts, top, device):
    i32 = dict(dtype=torch.int32, device=device)
    return R.Routing(torch.zeros((rows, top), **i32), torch.zeros((rows, top), device=device), torch.zeros(experts + 1, **i32),
                     torch.zeros(rows * top, **i32), torch.zeros((rows, top), **i32))


@pytest.mark.parametrize("missing", R.Routing._fields)
def test_a_missing_tensor_is_refused_first(missing):
    pkg_build.build()
    out = routing(3, 16, 4, "cpu")._replace(**{missing: None})
    with pytest.raises(ValueError, match="%s is needed" % missing):
        R.gemm_route_scored(torch.zeros((3, 16)), 4, out=out)


@pytest.mark.parametrize("out", [(), 5, [None] * 5, (None, None)])
def test_what_is_no_routing_is_refused(out):
    pkg_build.build()
    with pytest.raises(ValueError, match="out must be a Routing"):
        R.gemm_route_scored(torch.zeros((3, 16)), 4, out=out)


@pytest.mark.gpu
def test_a_routing_is_written_and_returned():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    z = torch.randn(40, 16, device="cuda")
    out = routing(40, 16, 4, "cuda")
    want = R.gemm_route_scored(z, 4, groups=4, top_groups=2)
    assert R.gemm_route_scored(z, 4, groups=4, top_groups=2, out=out) is out
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    for missing in R.Routing._fields:
        kept = [t.clone() for t in out]
        with pytest.raises(ValueError):
            R.gemm_route_scored(z + 1, 4, out=out._replace(**{missing: None}))
        with pytest.raises(ValueError):
            R.gemm_route_scored(z + 1, 4, out=out._replace(**{missing: torch.zeros(7, device="cuda")}))
        assert all(torch.equal(a, b) for a, b in zip(out, kept))
