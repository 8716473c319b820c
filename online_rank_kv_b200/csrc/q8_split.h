// Arithmetic of the split kernel's numbered-through steps (plain C++: the CPU
// test suite compiles it on its own).
#pragma once

#include <stdint.h>

#if defined(__CUDACC__)
#define ISKV_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define ISKV_HOST_DEVICE inline
#endif

namespace iskv {
namespace q8 {

// Where step `off` of a request lies, whose steps are numbered through (KV head,
// row tile, step).  The steps of one head pass 2^31 where many queries stand over
// a long request (two queries a tile: 371K tokens with as many queries).
struct StepPlace {
    int h, tile, step;
};

ISKV_HOST_DEVICE StepPlace place_of_step(int64_t off, int tiles, int steps) {
    const int64_t per_head = (int64_t)tiles * steps;
    StepPlace s;
    s.h = (int)(off / per_head);
    const int64_t rest = off - s.h * per_head;
    s.tile = (int)(rest / steps);
    s.step = (int)(rest - (int64_t)s.tile * steps);
    return s;
}

}  // namespace q8
}  // namespace iskv
