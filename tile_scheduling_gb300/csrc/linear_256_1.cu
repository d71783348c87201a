#include "linear_launch.cuh"

TS_LINEAR_VARIANT(linear_256_1, 256, 1, 0)
