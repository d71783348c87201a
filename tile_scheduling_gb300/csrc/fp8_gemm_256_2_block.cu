#include "fp8_launch.cuh"

TS_FP8_VARIANT(fp8_256_2_block, 256, 2, false, false, 128, 128)
