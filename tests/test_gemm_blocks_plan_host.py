"""Which kernel a product with block scales takes, as the library's own rule says on the CPU: the cases below reach each of the
large tiles, whole and with the sum over k in parts, with columns that end inside the second 128 of a tile of 256, so that
tests on the GPU can name the kernel that they cover (test_gpu_gemm_blocks_tiles.py).  A change of the rule that moves a case
elsewhere fails here."""
import ctypes

import pytest

dlf = pytest.importorskip("dl_fusion_amd", reason="libdlfusion.so not built")

TILE128, TILE128_DEEP, TILE256 = 5, 6, 7


class Args(ctypes.Structure):
    """GemmBlocksArgs of csrc/kernels.h."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("a", "a_scale", "b", "b_scale", "shift", "residual", "c")] + [("m", ctypes.c_int64)]
                + [(n, ctypes.c_int) for n in ("n", "k", "a_scale_stride", "b_scale_stride", "kind", "parts", "part_blocks", "part_stride")]
                + [("part", ctypes.c_void_p)])


def plan(m, n, k):
    """The kernel and the parts of the sum."""
    a = Args(m=m, n=n, k=k)
    dlf._lib._ZN3dlf16plan_gemm_blocksEPNS_14GemmBlocksArgsE(ctypes.byref(a))
    assert a.part_stride == -(-n // 4) * 4 and (a.parts - 1) * a.part_blocks < -(-k // 128) <= a.parts * a.part_blocks
    return a.kind, a.parts


# (kernel, sum in parts): columns whole 16 bytes of output, even, odd
CASES = {
    (TILE128, False): [(411, 7856, 1040), (399, 8178, 1040), (394, 7877, 1072)],
    (TILE128, True): [(65, 5056, 5600), (65, 3806, 7728), (67, 5027, 5360)],
    (TILE128_DEEP, False): [(199, 8368, 1056), (195, 8444, 1072), (194, 8943, 1088)],
    (TILE128_DEEP, True): [(65, 2704, 8688), (67, 4794, 5152), (69, 4239, 5536)],
    (TILE256, False): [(1057, 7376, 1040), (1425, 5542, 1040), (1586, 5089, 1088)],
    (TILE256, True): [(132, 5584, 8288), (130, 5578, 8336), (131, 5549, 8784)],
}


@pytest.mark.parametrize("kind,parts,size", [(kind, parts, size) for (kind, parts), sizes in CASES.items() for size in sizes])
def test_the_cases_reach_their_kernels(kind, parts, size):
    got = plan(*size)
    assert (got[0], got[1] > 1) == (kind, parts)
    m, n, k = size
    assert k > 8 * 128 and m % 16 and 128 < n % 256


def test_the_parts_are_those_of_the_workspace():
    for m, n, k in [s for sizes in CASES.values() for s in sizes] + [(1, 4096, 4096), (64, 4096, 11008), (8192, 4096, 11008)]:
        parts = plan(m, n, k)[1]
        assert dlf.dlf_gemm_blocks_workspace_bytes(dlf.gemm_blocks_desc(m, n, k)) == (parts * m * (-(-n // 4) * 4) * 4 if parts > 1 else 0)
