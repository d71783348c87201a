#include "linear_launch.cuh"

TS_LINEAR_VARIANT(linear_256_1_full, 256, 1, LIN_FULL)
