// santa_visible.cuh -- which keys a decode query sees: the first `sinks` of its sequence
// and the last `window`.
#pragma once

#include "santa_serving.h"

namespace santa {

struct Visible {
    int L;   // keys of the sequence
    int s;   // visible sinks
    int lo;  // first key of the window, >= s
};
__device__ __forceinline__ Visible visible(int L, int window, int sinks) {
    Visible v;
    v.L = L;
    v.s = min(sinks, L);
    v.lo = max(v.s, L - window);
    return v;
}

}  // namespace santa
