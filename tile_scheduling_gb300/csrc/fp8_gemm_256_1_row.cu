#include "fp8_launch.cuh"

TS_FP8_VARIANT(fp8_256_1_row, 256, 1, true, false, 256, 128)
