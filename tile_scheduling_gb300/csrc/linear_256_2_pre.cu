#include "linear_launch.cuh"

TS_LINEAR_VARIANT(linear_256_2_pre, 256, 2, LIN_PRE)
