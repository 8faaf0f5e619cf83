"""Every kernel instance of the 4-bit operators that the library holds is taken
by some call, and by a case that the GPU tests compare with the 64-bit
reference (no GPU needed here)."""
import mx4_instances as inst
import pytest

TYPES = (inst.F32, inst.BF16, inst.F16)


def test_product_cases_take_the_tiles_they_name():
    for shape, tile in inst.GEMMS.items():
        assert inst.gemm_tile(*shape) == tile
        assert inst.slabs(shape[2]) * 128 // tile[2] >= tile[5]          # at least as many chunks as stages
    assert set(inst.GEMMS) >= set(inst.ADDING)
    assert {inst.gemm_tile(*s) for s in inst.ADDING} == set(inst.GEMMS.values())
    for shape, tile in inst.STEPS.items():
        assert inst.gemm_pair(*shape) == tile


def test_products_reach_every_instance():
    assert inst.built("mx4_gemm_kernel") == {(*t, ty) for t in set(inst.GEMMS.values()) for ty in TYPES}
    assert inst.built("mx4_gemm_two_kernel") == {(*t, ty) for t in inst.STEPS.values() if t for ty in TYPES}


def test_thin_products_reach_every_instance():
    reached = {inst.linear_instance(ty, m, k) for ty in TYPES for m in inst.LINEAR_TOKENS for k in inst.LINEAR_COLS}
    assert inst.built("linear_kernel") == reached
    # and no other call takes another
    assert reached >= {inst.linear_instance(ty, m, 128 * n) for ty in TYPES for m in range(1, 65) for n in range(1, 80)}


@pytest.mark.parametrize("kernel", ["up_kernel", "down_kernel"])
def test_expert_layers_reach_every_instance(kernel):
    def of(t, top, hidden, inner):
        if kernel == "down_kernel":
            return [inst.down_instance(t, top, inner)]
        return [inst.up_instance(ty, t, top, hidden) for ty in TYPES]

    reached = set()
    for t, top in inst.EXPERT_TOKENS:
        for hidden in inst.EXPERT_HIDDEN:
            reached.update(of(t, top, hidden, 40))
        for inner in inst.EXPERT_INNER:
            reached.update(of(t, top, 48, inner))
    reached.discard(None)
    assert inst.built(kernel) == reached
    every = {i for t in range(1, 65) for top in range(1, 17) for n in range(1, 60) for i in of(t, top, 128 * n, 128 * n)}
    every.discard(None)
    assert reached == every
