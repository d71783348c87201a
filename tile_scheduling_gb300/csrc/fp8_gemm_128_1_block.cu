#include "fp8_launch.cuh"

TS_FP8_VARIANT(fp8_128_1_block, 128, 1, false, false, 128, 128)
