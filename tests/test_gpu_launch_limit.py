"""A launch that would need 2^32 threads or more in x is refused: the runtime takes
their number modulo 2^32 without an error, and most of the result stays unwritten."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("thin", ["columns", "rows"])
def test_more_workgroups_than_a_grid_takes(thin):
    """The thin kernels take 16 rows, or columns, to a workgroup of 512 threads."""
    import tiled_fp32_gemm_03_amd as g

    dev = torch.device("cuda:0")
    two = torch.full((1, 1), 2.0, device=dev)
    for n, fits in ((2 ** 27 - 16, True), (2 ** 27, False), (2 ** 27 + 40, False)):
        ones = torch.ones(n, device=dev)
        out = torch.zeros(n, device=dev)
        a, b, c = ((ones.view(n, 1), two, out.view(n, 1)) if thin == "columns"
                   else (two, ones.view(1, n), out.view(1, n)))
        if fits:
            g.matmul(a, b, out=c)
            right = bool((out == 2.0).all())
            assert right, n
        else:
            with pytest.raises(g.GemmError) as e:
                g.matmul(a, b, out=c)
            assert e.value.status == 5
