#include "linear_launch.cuh"

TS_LINEAR_VARIANT(linear_256_1_pre, 256, 1, LIN_PRE)
