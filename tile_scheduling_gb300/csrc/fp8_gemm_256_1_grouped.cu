#include "fp8_launch.cuh"

TS_FP8_VARIANT(fp8_256_1_grouped, 256, 1, false, true, 256, 128)
