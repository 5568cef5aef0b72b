"""Which kernel a product takes: the library's own rule, for tests that are there for one of its variants."""
import ctypes


class _Plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("stages", "per", "parts", "tm", "tn", "splits", "rows")]


def plan(M, N, K, parts=1):
    """C [M][N] over a reduction of K, A in `parts` parts: tiles' rows (256, 192 or 128) and splits."""
    import mixed_precision_bit_amd as lib
    f = lib._lib.lib()["_ZN3mpb11linear_planEllli"]  # mpb::linear_plan(int64, int64, int64, int)
    f.restype, f.argtypes = _Plan, [ctypes.c_int64] * 3 + [ctypes.c_int]
    p = f(M, N, K, parts)
    return p.rows, p.splits
