"""Every kernel instance of the 8-bit products and quantisations that the library holds is taken by some call, and by a
case that the GPU tests compare with exact sums (no GPU needed here)."""
import i8_instances as inst
import test_gpu_i8
import test_gpu_i8_instances as cases


def reached():
    all = set()
    for ty in inst.TYPES:
        for m, n, k in cases.PRODUCTS + test_gpu_i8.GEMMS:
            all |= inst.product(m, n, k, ty)
        for m, n, k in cases.THIN:
            all |= inst.product(m, n, k, ty) | inst.linear(m, n, k, ty)
        for m, n, k in test_gpu_i8.LINEARS + inst.PROMPTS:
            all |= inst.linear(m, n, k, ty)
        for m, n, k in cases.TRAINS + inst.STEPS + test_gpu_i8.TRAINS:
            all |= inst.backward(m, n, k, ty)
        for rows, cols in inst.COLUMNS:
            all |= inst.columns(rows, cols, ty)
        for rows, cols in test_gpu_i8.SHAPES:
            all |= inst.rows(cols, ty)
    return all


def test_cases_reach_every_instance():
    assert reached() == {(kernel, i) for kernel in inst.KERNELS for i in inst.built(kernel)}


def test_no_other_call_takes_another():
    sizes = [1, 8, 20, 40, 100, 200, 333, 700, 1100, 2100, 4100, 8200, 17000, 40000]
    every = set()
    for m in sizes:
        for n in sizes:
            for k in sizes:
                every |= inst.product(m, n, k, inst.BF16) | inst.linear(m, n, k, inst.BF16) | inst.backward(m, n, k, inst.BF16)
    assert every <= reached()


def test_steps_take_what_they_name():
    def alone(m, n, k):
        return {i[:6] for kernel, i in inst.backward(m, n, k, inst.BF16) if kernel == "i8_gemm_kernel" and i[7:] == (1, 1)}

    assert alone(*inst.STEPS[0]) == alone(*inst.STEPS[1]) == {inst.T128}
    m, n, _ = inst.STEPS[2]
    assert -(-m // 8) > 512 and n > 4096
    cut = [(inst.parts(m, k, inst.tile(m, k)), inst.parts(inst.piece_rows(n), k, inst.PAIRS[inst.tile(inst.piece_rows(n), k, True)]))
           for m, n, k in inst.STEPS[3:]]
    assert cut == [(True, False), (False, True), (True, True)]
    assert any(inst.parts(m, n, inst.tile(m, n)) for m, n, _ in cases.PRODUCTS)
