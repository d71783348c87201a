#include "fp8_launch.cuh"

TS_FP8_VARIANT(fp8_256_1_block, 256, 1, false, false, 256, 128)
