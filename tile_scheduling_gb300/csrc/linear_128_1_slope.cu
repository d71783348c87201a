#include "linear_launch.cuh"

TS_LINEAR_VARIANT(linear_128_1_slope, 128, 1, LIN_SLOPE)
