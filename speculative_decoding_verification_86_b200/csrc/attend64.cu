#define SV_ATTEND_WIDTH 64
#include "attend_launch.cuh"
