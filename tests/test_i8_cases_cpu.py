"""The GPU cases of the 8-bit products run every kernel that the dispatch can choose."""

from tests.i8_cases import EXPERTS, LINEAR, ROUTED, SHARED, ffn, one_pass

SIZES = (16, 100, 200, 400, 512, 800, 1000, 1600, 2048, 3000, 4096, 6144, 8200, 13000, 16400, 20000)
TOKENS = (1, 2, 3, 4, 5, 9, 16, 17, 30, 33, 64, 65, 129, 200, 300, 500, 800, 1000, 1400, 3000)


def test_linear_cases():
    every = {one_pass(T, 1, 1, False, N, K, False) for T in TOKENS for N in SIZES
             for K in (72, 9000)}
    assert {one_pass(T, 1, 1, False, N, K, False) for T, K, N in LINEAR} == every
    assert len(every) == 15


def test_shared_cases():
    every = {kern for T in TOKENS for H in SIZES for I in SIZES for kern in
             ffn(T, 1, 1, False, H, I)}
    assert {kern for c in SHARED for kern in ffn(c[0], 1, 1, False, *c[1:])} == every
    assert len(every) == 30


def test_routed_cases():
    every = {kern for T in TOKENS for E, k in ((2, 1), (5, 5), (12, 5), (64, 8), (256, 8), (1024, 16))
             for H in SIZES for I in SIZES for kern in ffn(T, k, E, True, H, I)}
    assert {kern for T, E, k, H, I in ROUTED for kern in ffn(T, k, E, True, H, I)} == every
    assert len(every) == 18


def test_many_experts_on_both_kernels():
    for most in (256, 300, 1024):
        kinds = {kern[0] for T, E, k, H, I, _ in EXPERTS if E == most
                 for kern in ffn(T, k, E, True, H, I)}
        assert kinds == {"streaming", "gemm"}
