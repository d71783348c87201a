#include "fp8_launch.cuh"

TS_FP8_VARIANT(fp8_128_1_row, 128, 1, true, false, 128, 128)
