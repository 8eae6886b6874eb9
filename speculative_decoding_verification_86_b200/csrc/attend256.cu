#define SV_ATTEND_WIDTH 256
#include "attend_launch.cuh"
