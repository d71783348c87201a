#include "fp8_launch.cuh"

TS_FP8_VARIANT(fp8_256_2_grouped, 256, 2, false, true, 128, 128)
