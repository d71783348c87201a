#include "linear_launch.cuh"

TS_LINEAR_VARIANT(linear_128_1, 128, 1, 0)
