#include "fp8_launch.cuh"

TS_FP8_VARIANT(fp8_128_1_grouped, 128, 1, false, true, 128, 128)
