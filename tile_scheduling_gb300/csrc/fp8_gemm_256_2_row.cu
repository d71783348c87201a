#include "fp8_launch.cuh"

TS_FP8_VARIANT(fp8_256_2_row, 256, 2, true, false, 128, 128)
