#include "linear_launch.cuh"

TS_LINEAR_VARIANT(linear_256_2, 256, 2, 0)
