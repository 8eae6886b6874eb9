#define SV_ATTEND_WIDTH 128
#include "attend_launch.cuh"
