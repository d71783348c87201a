#include "linear_launch.cuh"

TS_LINEAR_VARIANT(linear_256_2_slope, 256, 2, LIN_SLOPE)
