"""Batches of the 4-bit products by the kernel that runs them: the mean rows an expert on
both sides of each rule.  tests/test_int4_kernels_cpu.py holds them to the library's rule,
tests/test_gpu_int4_kernels.py runs them."""

E, K = 4, 2                                              # experts, slots a token
LONG = 4608                                              # 36 blocks of 128 columns: a wave of four has 8 or 10

# (mode, group, mean): kernel
KERNELS = {}
for group in (32, 64, 128):
    up, down = (30, 22) if group == 32 else (26, 17)
    for mode, tiles in (("gate_up", up), ("down", down)):
        for mean in (1, 13):
            KERNELS[mode, group, mean] = "rows16"
        for mean in (14, 15, tiles - 1):
            KERNELS[mode, group, mean] = "rows32"
        for mean in (tiles, 40):
            KERNELS[mode, group, mean] = "tiles"


def batch(mode, mean):
    """(T, D, F, Fs): mean rows an expert, a long reduction, 256 outputs, a shared expert"""
    return (mean * E // K, LONG, 256, 256) if mode == "gate_up" else (mean * E // K, 256, LONG, LONG)
